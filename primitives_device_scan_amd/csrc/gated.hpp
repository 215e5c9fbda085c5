// gated.hpp -- what the gated recurrence and its gradient share: a scan over
// packed rows whose steps are pairs (a, b), (a, b) and then (a', b') being
// (a a', a' b + b').
//
// The rows are cut into tiles whatever the sequences' lengths are. A workgroup
// holds a tile of kSub * TQ rows by kLanes * V channels in registers, read once:
// 16 lanes hold TQ successive rows of 16 V channels, V to a lane. A tile makes
// its pair (A, B), publishes it, and finds the state that enters it from the
// pairs of the tiles before it in its group and the state that entered the group,
// which the group before published. Which pairs are joined is fixed by the
// positions, so results do not depend on which tile was first. A sequence's
// first row starts anew: a tile that has one needs no earlier state behind it.
//
// Words between workgroups are 64 bits, a value and a mark of what it is, so
// that a value needs no order with a flag; a launch before clears them. Tile t
// waits for lower tiles only, which are dispatched before it, and every wait
// ends after the spin limit (the state is NaN then).
#pragma once

#include <type_traits>

#include "float_types.hpp"
#include "gate.hpp"
#include "launch.hpp"

namespace ds {


constexpr int kLanes = 16;                              // lanes side by side in a row
constexpr int kSub = kThreads / kLanes;                 // parts of a tile's rows
constexpr int kGroup = 8;                               // tiles to a group
constexpr uint32_t kPair = 1, kState = 2;               // marks: a pair (A, B), or B alone, a state

// V elements of T at any element alignment, as they lie in memory. An address
// is a row that all lanes have in common and a lane's bytes from it (32 bits:
// kMostStride), so that a tile's many addresses take scalar registers.
template <typename T, int V> struct Cells {
    typename std::conditional<V == 1, T, u32x4>::type raw;
    using At = typename std::conditional<V == 1, T, typename Vec16<T>::type>::type;
    __device__ __forceinline__ void load(const T* row, uint32_t bytes)
    {
        raw = *reinterpret_cast<const At*>(reinterpret_cast<const char*>(row) + bytes);
    }
    __device__ __forceinline__ void store(T* row, uint32_t bytes) const
    {
        *reinterpret_cast<At*>(reinterpret_cast<char*>(row) + bytes) = raw;
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
        if constexpr (V != 1) asm volatile("" : "+v"(raw));
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

__device__ __forceinline__ uint64_t marked(uint32_t mark, float v)
{
    return (uint64_t)mark << 32 | __builtin_bit_cast(uint32_t, v);
}

// The state that enters tile `tile` in this thread's channel, from the words of
// the tiles before it. `pairs`, `entries`: this channel's words, of the pairs
// (two) and of the states that enter groups; `step` words to the next tile's.
__device__ __forceinline__ float entering_state(uint64_t* pairs, uint64_t* entries, int64_t step, int64_t tile,
                                                uint32_t spin_limit)
{
    constexpr int kBatch = 4;
    const int64_t group = tile / kGroup;
    uint32_t polls = 0;
    float a = 1.0f, b = 0.0f;  // the steps from after tile j up to this one
    for (int64_t j = tile - 1; j >= group * kGroup; j -= kBatch) {
        uint64_t wa[kBatch], wb[kBatch];
        for (;;) {
            bool ready = true;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t at = max(j - i, group * kGroup) * step;
                wa[i] = status_load(pairs + 2 * at);
                wb[i] = status_load(pairs + 2 * at + 1);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                ready &= (uint32_t)(wb[i] >> 32) == kState || ((wa[i] >> 32) && (wb[i] >> 32));
            if (ready) break;
            if (++polls >= spin_limit) return __builtin_nanf("");
            __builtin_amdgcn_s_sleep(1);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (j - i < group * kGroup) break;
            b = __builtin_fmaf(a, __builtin_bit_cast(float, (uint32_t)wb[i]), b);
            if ((uint32_t)(wb[i] >> 32) == kState) return b;
            a *= __builtin_bit_cast(float, (uint32_t)wa[i]);
        }
    }
    for (;;) {
        const uint64_t w = status_load(entries + group * step);
        if (w >> 32) return __builtin_fmaf(a, __builtin_bit_cast(float, (uint32_t)w), b);
        if (++polls >= spin_limit) return __builtin_nanf("");
        __builtin_amdgcn_s_sleep(1);
    }
}

// From the parts' pairs in s_a, s_b (s_new: the part starts anew) to the state
// that enters each part, which replaces its A. `needs`: a state enters the tile.
template <int SPAN>
__device__ __forceinline__ void join_parts(float (&s_a)[kSub][SPAN], float (&s_b)[kSub][SPAN], const int (&s_new)[kSub],
                                           int64_t tile, int64_t tiles, int64_t cblock, int64_t cblocks, bool needs,
                                           const GatedWords& w)
{
    const int i = (int)threadIdx.x;
    if (i >= SPAN) return;
    float a = 1.0f, b = 0.0f;
    bool anew = false;
#pragma unroll 4
    for (int q = 0; q < kSub; ++q) {
        b = s_new[q] ? s_b[q][i] : __builtin_fmaf(s_a[q][i], b, s_b[q][i]);
        a *= s_a[q][i];
        anew |= s_new[q] != 0;
    }
    const int64_t step = cblocks * SPAN;
    uint64_t* const pairs = w.pairs + 2 * (cblock * SPAN + i);
    uint64_t* const entries = w.entries + cblock * SPAN + i;
    float h = 0.0f;
    if (tiles > 1) {
        uint64_t* const mine = pairs + 2 * tile * step;
        if (!anew) status_store(mine, marked(kPair, a));
        status_store(mine + 1, marked(anew ? kState : kPair, b));
        if (needs) h = entering_state(pairs, entries, step, tile, w.spin_limit);
        if (tile % kGroup == kGroup - 1 && tile + 1 < tiles)
            status_store(entries + (tile / kGroup + 1) * step, marked(kState, anew ? b : __builtin_fmaf(a, h, b)));
    }
#pragma unroll 4
    for (int q = 0; q < kSub; ++q) {
        const float to = s_new[q] ? s_b[q][i] : __builtin_fmaf(s_a[q][i], h, s_b[q][i]);
        s_a[q][i] = h;
        h = to;
    }
}

// The sequences of rows row0 - 1 .. row0 + ROWS into s_seq; true if they are all
// the same one.
template <int ROWS>
__device__ __forceinline__ bool find_sequences(const GatedScan& a, int64_t row0, int (&s_seq)[ROWS + 2])
{
    const int first = sequence_of(a, row0 - 1);
    bool same = first >= 0;
    for (int i = threadIdx.x; i < ROWS + 2; i += kThreads) {
        const int s = sequence_of(a, row0 - 1 + i);
        s_seq[i] = s;
        same &= s == first;
    }
    return __syncthreads_and(same);
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

// Rows of a part: what the registers hold at two workgroups to a CU.
template <typename T> constexpr int kScanRows = sizeof(T) == 4 ? 16 : 12;
template <typename T> constexpr int kGradRows = 8;

inline int vector_of(ElemKind kind, int64_t dim)
{
    const int v = kind == kF32 ? 4 : 8;
    return dim < v ? 1 : v;
}

inline GatedPlan gated_plan_of(ElemKind kind, bool grad, int64_t tokens, int64_t dim)
{
    const int64_t rows = kSub * (grad ? (kind == kF32 ? kGradRows<float> : kGradRows<bf16>)
                                       : (kind == kF32 ? kScanRows<float> : kScanRows<bf16>)),
                  span = (int64_t)kLanes * vector_of(kind, dim);
    GatedPlan p;
    p.tiles = tokens > 0 ? (tokens + rows - 1) / rows : 1;
    p.cblocks = (dim + span - 1) / span;
    p.pair_words = p.tiles > 1 ? 2 * p.tiles * p.cblocks * span : 0;
    p.words = p.tiles > 1 ? p.pair_words + (p.tiles + kGroup - 1) / kGroup * p.cblocks * span : 0;
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


// The words of a call in its scratch, cleared.
GatedWords clear_words(const GatedPlan& plan, uint64_t* scratch, uint32_t spin_limit, hipStream_t stream);

}  // namespace ds
