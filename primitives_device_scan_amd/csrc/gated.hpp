// gated.hpp -- what the gated recurrence and its gradient share: a scan over
// packed rows whose steps are pairs (a, b), (a, b) and then (a', b') being
// (a a', a' b + b').
//
// The rows are cut into tiles whatever the sequences' lengths are. A workgroup
// holds a tile of kSub * TQ rows by kLanes * V channels in registers, read once:
// 16 lanes hold TQ successive rows of 16 V channels, V (16 bytes) to a lane. A tile makes
// its pair (A, B), publishes it, and finds the state that enters it from the
// pairs of the tiles before it in its group and the state that entered the group,
// which the group before published. Which pairs are joined is fixed by the
// positions, so results do not depend on which tile was first. A sequence's
// first row starts anew: a tile that has one needs no earlier state behind it.
// Tiles of one sequence alone are held in registers; of a tile in which sequences
// meet, the rows are read a second time, two or four at a time, which costs few
// registers (the same code for both needed more than there are and spilled).
//
// A scan has 3 elements' bytes a step (gate, x, h), its gradient 5 or, mixed, 6, and
// some 10 to 20 operations: memory is the floor. What keeps it from that floor:
// 2,028 vector instructions a wave, which fill half of its time, and the tiles'
// waits for each other (65,536 x 2,048 of 32 sequences in bf16, sigmoid, mixed: 227
// us, 3.5 TB/s; 186 with the waits left out, 129 at a copy's rate; the gradient of
// 32,768 x 4,096, one sequence: 350 us, 4.6 TB/s; 258; in fp32 32,768 x 2,048 of 16
// sequences 184 and 332 us, 4.4 and 4.9 TB/s). Of few channels the chain of groups is
// the time (65,536 x 64, one sequence: 123 us, where the bytes take 4).
//
// Words between workgroups are 64 bits, a pair or a state and which of them it is
// in one, so that a value needs no order with a flag; a launch before clears them
// and finds each tile's sequence. A wave waits with one lane to an earlier tile
// and reads all its channels' words once they are there (each channel polling its
// own words kept the fabric busy: one sequence of 65,536 rows by 2,048 channels 243 us
// instead of 203). Tile t waits for lower tiles only, which are dispatched before
// it, and every wait ends after the spin limit (the state is NaN then, and `gave_up` set).
#pragma once

#include <type_traits>

#include "float_types.hpp"
#include "gate.hpp"
#include "launch.hpp"

namespace ds {


constexpr int kLanes = 16;                              // lanes side by side in a row
constexpr int kSub = kThreads / kLanes;                 // parts of a tile's rows
constexpr int kGroup = 8;                               // tiles to a group

// V elements of T at any element alignment, as they lie in memory. An address
// is a row that all lanes have in common and a lane's bytes from it (32 bits:
// kMostStride), so that a tile's many addresses take scalar registers.
template <typename T, int V> struct Cells {
    static constexpr int kBytes = V * (int)sizeof(T);  // 16, 4 or an element
    typename std::conditional<kBytes == 16, u32x4, typename std::conditional<kBytes == 4, uint32_t, T>::type>::type raw;
    __device__ __forceinline__ void load(const T* row, uint32_t bytes)
    {
        const char* const p = reinterpret_cast<const char*>(row) + bytes;
        if constexpr (kBytes == 16)
            raw = *reinterpret_cast<const typename Vec16<T>::type*>(p);
        else
            __builtin_memcpy(&raw, reinterpret_cast<const T*>(p), kBytes);
    }
    __device__ __forceinline__ void store(T* row, uint32_t bytes) const
    {
        char* const p = reinterpret_cast<char*>(row) + bytes;
        if constexpr (kBytes == 16)
            *reinterpret_cast<typename Vec16<T>::type*>(p) = raw;
        else
            __builtin_memcpy(reinterpret_cast<T*>(p), &raw, kBytes);
    }
    __device__ __forceinline__ void fill(T x)
    {
        T t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = x;
        __builtin_memcpy(&raw, t, sizeof(t));
    }
    __device__ __forceinline__ void put(int k, T x)
    {
        T t[V];
        __builtin_memcpy(t, &raw, sizeof(t));
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = i == k ? x : t[i];
        __builtin_memcpy(&raw, t, sizeof(t));
    }
    __device__ __forceinline__ float operator[](int i) const
    {
        T t[V];
        __builtin_memcpy(t, &raw, sizeof(t));
        return (float)t[i];
    }
    __device__ __forceinline__ void set(const float (&x)[V])
    {
        T t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = (T)x[i];
        __builtin_memcpy(&raw, t, sizeof(t));
    }
    // What was worked out of it before is not kept for later: the registers are
    // for the rows themselves.
    __device__ __forceinline__ void pin()
    {
        if constexpr (kBytes == 16) asm volatile("" : "+v"(raw));
    }
};
template <int V>
__device__ __forceinline__ void pin(float (&x)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) asm volatile("" : "+v"(x[i]));
}
template <int V>
__device__ __forceinline__ void load_states(const float* p, float (&x)[V])
{
    __builtin_memcpy(x, p, sizeof(x));
}
template <int V>
__device__ __forceinline__ void store_states(float* p, const float (&x)[V])
{
    __builtin_memcpy(p, x, sizeof(x));
}

// The sequence that row t belongs to, or -1.
__device__ __forceinline__ int sequence_of(const GatedScan& a, int64_t t)
{
    if (t < 0 || t >= a.tokens) return -1;
    if (!a.offsets) return 0;
    int64_t lo = 0, hi = a.sequences;  // the last s with offsets[s] <= t, if there is one
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.offsets[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return a.offsets[lo] <= t && t < a.offsets[lo + 1] ? (int)lo : -1;
}

// Where a workgroup's tile and channels are. Channels are counted in slots: the
// last lane with channels in the row takes the row's last V, some of them also
// its neighbour's, which then works them out twice, alike.
template <int V> struct Place {
    int64_t tile, cblocks, cblock, channel, slot;
    bool live;  // this lane has channels
    __device__ __forceinline__ Place(int64_t dim)
    {
        constexpr int kSpan = kLanes * V;
        cblocks = (dim + kSpan - 1) / kSpan;
        tile = blockIdx.x / cblocks;
        cblock = blockIdx.x % cblocks;
        slot = cblock * kSpan + (int)(threadIdx.x % kLanes) * V;
        live = slot < dim;
        channel = min(slot, dim - V);
    }
};

// A matrix as a tile sees it: row k of every part.
template <typename T> struct Rows {
    T* row;          // the tile's first (the gradient's h: the one before)
    int64_t stride;  // elements
    uint32_t bytes;  // from there to this lane's part and channels
    __device__ __forceinline__ Rows(T* p, int64_t s, int64_t row0, int part_row, int64_t channel)
        : row(p + row0 * s), stride(s), bytes((uint32_t)((part_row * s + channel) * (int64_t)sizeof(T)))
    {
    }
    __device__ __forceinline__ T* at(int k) const { return row + k * stride; }
};

// A word: 0 while there is nothing, else B and above it A (no NaN but one, its
// bits turned by kTurn, so that they are never 0), or kState and a state.
constexpr uint32_t kTurn = 0x7fffffffu, kState = 1;
__device__ __forceinline__ uint64_t pair_word(float a, float b)
{
    const uint32_t bits = a == a ? __builtin_bit_cast(uint32_t, a) : 0x7fc00000u;
    return (uint64_t)(bits ^ kTurn) << 32 | __builtin_bit_cast(uint32_t, b);
}
__device__ __forceinline__ uint64_t state_word(float h) { return (uint64_t)kState << 32 | __builtin_bit_cast(uint32_t, h); }
__device__ __forceinline__ float first_of(uint64_t w) { return __builtin_bit_cast(float, (uint32_t)(w >> 32) ^ kTurn); }
__device__ __forceinline__ float second_of(uint64_t w) { return __builtin_bit_cast(float, (uint32_t)w); }

// Set where a wait gives up; of this file's kernels, on each GPU.
static __device__ uint32_t gave_up;
// On the host: whether a wait gave up on the current GPU since the last time (sets *flag if so).
static hipError_t take_give_up(bool* flag)
{
    uint32_t set = 0;
    hipError_t e = hipMemcpyFromSymbol(&set, HIP_SYMBOL(gave_up), sizeof(set));
    if (e != hipSuccess || !set) return e;
    *flag = true;
    set = 0;
    return hipMemcpyToSymbol(HIP_SYMBOL(gave_up), &set, sizeof(set));
}

// The state that enters tile `tile` in this thread's channel, from the words of
// the tiles before it in its group and of the group; all lanes of a wave call
// it. `pairs`, `entries`: this channel's words, `step` words to the next tile's.
// polls: spin_limit after a wait that gave up, else less.
template <GateForm FORM>
__device__ __forceinline__ float entering_state(uint64_t* pairs, uint64_t* entries, int64_t step, int64_t tile,
                                                uint32_t spin_limit, uint32_t& polls)
{
    const int lane = lane_id();
    const int64_t group = tile / kGroup;
    const int before = (int)(tile - group * kGroup);  // tiles of the group; word `before` is the group's own
    // lane l: word l of the wave's first channel
    uint64_t* const first = reinterpret_cast<uint64_t*>(readlane((uint64_t)(uintptr_t)pairs, 0));
    uint64_t* const entry = reinterpret_cast<uint64_t*>(readlane((uint64_t)(uintptr_t)entries, 0));
    uint64_t* const mine = lane < before ? first + (tile - 1 - lane) * step : entry + group * step;
    int need;  // words 0 .. need: up to the first state
    for (;;) {
        const uint32_t mark = lane <= before ? (uint32_t)(status_load(mine) >> 32) : kState;
        const uint64_t there = ballot(mark != 0), states = ballot(mark == kState);
        need = min(before, __builtin_ctzll(states | (uint64_t)1 << before));
        const uint64_t wanted = ((uint64_t)2 << need) - 1;
        if ((there & wanted) == wanted) break;
        if (++polls >= spin_limit) return __builtin_nanf("");
        __builtin_amdgcn_s_sleep(1);
    }
    uint64_t w[kGroup] = {};
    for (;;) {
        bool there = true;
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
            if (i <= need) w[i] = status_load(i < before ? pairs + (tile - 1 - i) * step : entries + group * step);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) there &= i > need || (w[i] >> 32) != 0;
        if (ballot(!there) == 0) break;
        if (++polls >= spin_limit) return __builtin_nanf("");
    }
    float h = 0.0f;
#pragma unroll
    for (int i = kGroup - 1; i >= 0; --i)
        if (i <= need)
            h = (uint32_t)(w[i] >> 32) == kState ? second_of(w[i]) : keep_of<FORM>(first_of(w[i]), h) + second_of(w[i]);
    return h;
}

// Where a tile's first row's state comes from.
enum Enter { kNone, kGiven, kBefore };  // nowhere (all parts' states are their own), `given`, the tile before

// From the parts' pairs in s_a (as Product has them), s_b (s_new: the part starts anew) to the state
// that enters each part, which replaces its A. `given`: a state for each channel,
// or null for 0.
template <int V, GateForm FORM>
__device__ __forceinline__ void join_parts(float (&s_a)[kSub][kLanes * V], float (&s_b)[kSub][kLanes * V],
                                           const int (&s_new)[kSub], const Place<V>& p, int64_t tiles, int64_t dim,
                                           Enter enter, const float* given, const GatedWords& w)
{
    constexpr int kSpan = kLanes * V;
    const int i = (int)threadIdx.x;
    if (i >= kSpan) return;
    Product<FORM> all;
    float b = 0.0f, h = 0.0f;
    if (enter == kGiven && given) h = given[min(p.cblock * kSpan + i / V * V, dim - V) + i % V];
    bool anew = false;
#pragma unroll 4
    for (int q = 0; q < kSub; ++q) {
        b = (s_new[q] ? 0.0f : keep_of<FORM>(s_a[q][i], b)) + s_b[q][i];
        all.step(s_a[q][i]);
        anew |= s_new[q] != 0;
    }
    if (tiles > 1) {
        const int64_t step = p.cblocks * kSpan;
        uint64_t* const pairs = w.pairs + p.cblock * kSpan + i;
        uint64_t* const entries = w.entries + p.cblock * kSpan + i;
        const bool known = anew || enter == kGiven;  // what leaves does not depend on the tiles before
        const float a = all.value(), leaving = anew ? b : keep_of<FORM>(a, h) + b;
        status_store(pairs + p.tile * step, known ? state_word(leaving) : pair_word(a, b));
        uint32_t polls = 0;
        if (enter == kBefore) h = entering_state<FORM>(pairs, entries, step, p.tile, w.spin_limit, polls);
        if (p.tile % kGroup == kGroup - 1 && p.tile + 1 < tiles)
            status_store(entries + (p.tile / kGroup + 1) * step,
                         state_word(known ? leaving : keep_of<FORM>(a, h) + b));
        if (polls >= w.spin_limit) __hip_atomic_store(&gave_up, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll 4
    for (int q = 0; q < kSub; ++q) {
        const float to = (s_new[q] ? 0.0f : keep_of<FORM>(s_a[q][i], h)) + s_b[q][i];
        s_a[q][i] = h;
        h = to;
    }
}

// A tile's one sequence, or none (-1: sequences meet in it, or it has rows of
// none), and whether it begins at the tile's first row and ends at its last.
struct TileInfo {
    int32_t sequence;
    uint32_t ends;  // 1: begins here, 2: ends here
};
__device__ __forceinline__ TileInfo tile_info(const GatedScan& a, int64_t row0, int rows)
{
    const int64_t last = min(row0 + rows, a.tokens) - 1;
    const int s = sequence_of(a, row0), before = sequence_of(a, row0 - 1), after = sequence_of(a, last + 1);
    TileInfo t;
    t.sequence = s >= 0 && sequence_of(a, last) == s ? s : -1;
    t.ends = (before != s ? 1u : 0u) | (after != s ? 2u : 0u);
    return t;
}
// ... from the launch before, or of the only tile
__device__ __forceinline__ TileInfo info_of(const GatedScan& a, const GatedWords& w, int64_t tiles, int64_t at, int rows)
{
    TileInfo t;
    if (tiles > 1)
        t = reinterpret_cast<const TileInfo*>(w.infos)[at];
    else
        t = tile_info(a, 0, rows);
    t.sequence = __builtin_amdgcn_readfirstlane(t.sequence);
    if (t.sequence >= a.sequences) t.sequence = -1;  // it indexes the states: never past them
    t.ends = (uint32_t)__builtin_amdgcn_readfirstlane((int)t.ends);
    return t;
}

// A gate that keeps the state as it is, for rows past the end.
template <typename T, GateForm FORM> __device__ __forceinline__ T open_gate()
{
    return (T)(FORM == kSigmoid ? __builtin_inff() : FORM == kLog ? 0.0f : 1.0f);
}

// The sequences of rows row0 - 1 .. row0 + ROWS into s_seq.
template <int ROWS>
__device__ __forceinline__ void find_sequences(const GatedScan& a, int64_t row0, int (&s_seq)[ROWS + 2])
{
    for (int i = threadIdx.x; i < ROWS + 2; i += kThreads) s_seq[i] = sequence_of(a, row0 - 1 + i);
    __syncthreads();
}

// Sequences without rows: `to` gets `from`, or 0.
template <int V>
__device__ __forceinline__ void pass_empty(const GatedScan& a, const Place<V>& p, const float* from, float* to)
{
    if ((!a.offsets && a.tokens > 0) || !to || !p.live) return;
    const int64_t tiles = gridDim.x / p.cblocks;
    for (int64_t s = p.tile * kSub + threadIdx.x / kLanes; s < a.sequences; s += tiles * kSub) {
        if (a.tokens > 0) {
            const int64_t first = min(max((int64_t)a.offsets[s], (int64_t)0), a.tokens);
            if (min((int64_t)a.offsets[s + 1], a.tokens) > first) continue;
        }
        float x[V] = {};
        if (from) load_states(from + s * a.dim + p.channel, x);
        store_states(to + s * a.dim + p.channel, x);
    }
}

// Rows of a part, by what the registers hold: of the scan 8 at three workgroups to a
// CU (65,536 x 2,048: 227 us; 4 rows 247, four workgroups of 6 rows 228); of the
// gradient of mixed inputs in 16 bits, which holds four matrices, 4 at three
// workgroups (32,768 x 4,096: 351 us, 8 rows at two 396), of other gradients 8 at two.
template <typename T> constexpr int kScanRows = 8;
template <typename T, bool MIX> constexpr int kGradRows = sizeof(T) == 2 && MIX ? 4 : 8;
template <typename T, bool MIX> constexpr int kGradPerCu = sizeof(T) == 2 && MIX ? 3 : 2;

inline int vector_of(ElemKind kind, int64_t dim)
{
    const int v = kind == kF32 ? 4 : 8;
    return dim < v ? 1 : v;
}

// Workgroups of 16 bytes to a lane below which a lane has 4 instead: four times as
// many, each of a quarter of the work (256 rows of four sequences by 2,048 channels
// in bf16, 32 workgroups: 18.5 us, 14.6 so; the gradient of 1,003 x 1,000 in fp32,
// 128 workgroups: 19.1 and 19.6).
constexpr int64_t kNarrowBelow = 128;

inline GatedPlan gated_plan_of(ElemKind kind, bool grad, bool mix, int64_t tokens, int64_t dim)
{
    const int part = !grad              ? (kind == kF32 ? kScanRows<float> : kScanRows<bf16>)
                     : kind == kF32 ? (mix ? kGradRows<float, true> : kGradRows<float, false>)
                                    : (mix ? kGradRows<bf16, true> : kGradRows<bf16, false>);
    const int64_t rows = kSub * part;
    GatedPlan p;
    p.tiles = tokens > 0 ? (tokens + rows - 1) / rows : 1;
    p.vector = vector_of(kind, dim);
    const auto blocks = [&] { return (dim + kLanes * p.vector - 1) / (kLanes * p.vector); };
    if (p.tiles * blocks() < kNarrowBelow) p.vector = kind == kF32 || dim < 2 ? 1 : 2;
    p.cblocks = blocks();
    const int64_t span = (int64_t)kLanes * p.vector;
    p.pair_words = p.tiles > 1 ? p.tiles * p.cblocks * span : 0;
    p.rows = rows;
    p.entry_words = p.tiles > 1 ? (p.tiles + kGroup - 1) / kGroup * p.cblocks * span : 0;
    p.words = p.tiles > 1 ? p.pair_words + p.entry_words + p.tiles : 0;
    return p;
}

template <typename F> void with_form(int form, bool mix, F&& f)
{
    const auto go = [&](auto fm) {
        if (mix)
            f(fm, std::true_type{});
        else
            f(fm, std::false_type{});
    };
    if (form == kDecay)
        go(std::integral_constant<GateForm, kDecay>{});
    else if (form == kLog)
        go(std::integral_constant<GateForm, kLog>{});
    else
        go(std::integral_constant<GateForm, kSigmoid>{});
}

template <typename F> hipError_t with_type(ElemKind kind, int form, bool mix, F&& f)
{
    with_form(form, mix, [&](auto fm, auto mx) {
        if (kind == kF32)
            f(float{}, fm, mx);
        else if (kind == kBF16)
            f(bf16{}, fm, mx);
        else
            f(fp16{}, fm, mx);
    });
    return hipGetLastError();
}

// f(a lane's channels) of a plan: those of 16 bytes, of 4, or one
template <typename T, typename F> void with_vector(int vector, F&& f)
{
    if (vector == Vec16<T>::kN)
        f(std::integral_constant<int, Vec16<T>::kN>{});
    else if (vector == 1)
        f(std::integral_constant<int, 1>{});
    else if constexpr (sizeof(T) == 2)
        f(std::integral_constant<int, 2>{});
}

// The words of a call in its scratch, cleared, and its tiles' sequences.
GatedWords begin_words(const GatedScan& a, const GatedPlan& plan, uint64_t* scratch, uint32_t spin_limit,
                       hipStream_t stream);

}  // namespace ds
