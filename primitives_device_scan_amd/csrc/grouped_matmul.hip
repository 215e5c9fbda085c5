// grouped_matmul.hip -- matrix products grouped by expert: rows [offsets[e],
// offsets[e + 1]) of a batch belong to expert e,
//
//   y_r = W_e x_r   or, transposed, y_r = W_e^T x_r          W_e: rows x cols
//   dW_e = sum over its rows r of dy_r x_r^T
//
// Row r of the batch is row r of x, or, with an index, row index[r] / top_k of
// it (zeros where that is no row): the batch that the MoE alignment orders.
//
// All three are C[m, n] = sum over k of A[m, k] B[n, k], with operands whose
// memory runs along k (rows of the batch, rows of W) or across it (W transposed,
// both operands of dW, whose k are rows of the batch). A workgroup of four waves
// makes a tile of C, 2 x 2 waves of TM x TN blocks of 32 x 32 (the matrix
// instructions' 32 x 32 x 16), from stages of 32 k in LDS.
//
// Operands whose rows start on 16 bytes and whose lengths are whole segments of
// 16 bytes go to LDS by loads that write it directly, three stages ahead of the
// one that is multiplied, in one stream over all of a workgroup's tiles. One
// barrier to a stage; the reads of the next 16 k lie between the matrix
// instructions of the last. Other operands go through registers (RowsOdd).
//
// In LDS an operand along k has 64 bytes of each row, row r's segment s at
// s ^ (r / 2) mod 4; one across k has lines of all rows, line k's segment s at
// s ^ 2 (k mod 4), and is turned as it is read (ds_read_b64_tr_b16). In both
// orders the lanes that are served together lie in different banks.
//
// Bound by the matrix cores for many rows: 65,536 rows of 64 experts, 1,536 x 2,048
// in bf16, run at 880 to 917 TFLOP/s (449-467 us; a large plain product 1,163), the
// gradient of the matrices, indexed, at 764 to 790 (522-540 us): the matrix
// instructions are busy for 0.50 and 0.32 of the cycles, what is left are the tiles'
// starts and ends and the waits at a stage's barrier, and the gradient turns both its
// operands as it reads them. For few rows it is the matrices' bytes (256 experts of
// that size with some 8, 32, 128 rows each: 348-361, 361-376, 417-419 us; the bytes 258).
//
// Workgroups stay and take one tile after another; each finds the experts' tiles
// by a prefix sum of its own over the groups. Workgroup i runs on XCD i % 8: each
// XCD takes a contiguous run of tiles, so that what its tiles share is in its L2.
#include <type_traits>
#include <utility>

#include "float_types.hpp"
#include "launch.hpp"

namespace ds {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

template <typename T>
__device__ __forceinline__ f32x16 mma32(const u32x4& a, const u32x4& b, f32x16 c)
{
    if constexpr (__is_same(T, bf16))
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
}

constexpr int kDepth = 32;           // k of a stage
constexpr int kBlockBytes = 4096;    // of a stage, for 64 rows of an operand
constexpr int kRing = 4;             // stages in LDS
constexpr int kMostGroups = 2048;
// Rows of a batch, tiles' rows past a group's end and stages past its depth (up to
// kAhead + 1 of them) are counted in 32 bits: the host takes 2^31 - 512 rows at most.
constexpr int kXcds = 8;

// What lanes that have nothing to load read instead.
static __device__ __align__(16) uint32_t zeros[128];  // a line of a tile


__device__ __forceinline__ void group_range(const Grouped& a, int e, int64_t& first, int64_t& end)
{
    first = min(max((int64_t)a.offsets[e], (int64_t)0), a.m);
    end = min(max((int64_t)a.offsets[e + 1], first), a.m);
}

// The row of x that an entry of the index names, or -1; entry / top_k by a
// product (for 0 <= n < 2^31).
__device__ __forceinline__ int32_t row_of_entry(const Grouped& a, int32_t i)
{
    const uint32_t n = (uint32_t)i, t = (n + __umulhi(n, a.magic)) >> a.shift;
    return n < a.entries ? (int32_t)t : -1;
}
__device__ __forceinline__ int64_t batch_row(const Grouped& a, int64_t r)
{
    return a.index ? row_of_entry(a, a.index[r]) : r;
}

// This lane's 8 k of one row: of block `b` of 32 rows from `first` on, half `kk`
// of the stage, from an operand of 64 R rows.
template <int R, bool ACROSS>
__device__ __forceinline__ u32x4 read_fragment(const lds_char* stage, int first, int b, int kk, int lane)
{
    if constexpr (!ACROSS) {
        const int r = first + lane % 32;
        return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(
            stage + r * 64 + (((kk * 2 + lane / 32) ^ (r >> 1)) & 3) * 16 + b * 32 * 64);
    } else {
        // of 16 lanes, lanes 4 j .. 4 j + 3 name 16 rows of line j, and each lane
        // receives what four lines have of its own row
        const int j = lane % 16 / 4, line = kk * 16 + lane / 32 * 8 + j;
        const int row = first + 32 * b + lane / 16 % 2 * 16 + lane % 4 * 4;
        const lds_char* const at = stage + line * (128 * R) + (row / 8 ^ j * 2) * 16 + row % 8 * 2;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 4 * 128 * R));
        u32x4 v;
        __builtin_memcpy(&v, &lo, 8);
        __builtin_memcpy(reinterpret_cast<char*>(&v) + 8, &hi, 8);
        return v;
    }
}

enum GroupedOp { kProduct = 0, kTransposed = 1, kGradient = 2 };

// A tile of C and where its operands are.
struct Tile {
    int m0, n0;           // in y: row of the batch, column; in dW_e: row, column
    int e, first, end;    // the expert and its rows
    int depth;
    bool there;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The tiles of this workgroup: every `step`-th of [at, end).
struct Turns {
    int at, end, step;
};

// s_first[e] = the sum of of_rows(group's rows) over the groups before e; returns
// that over all. Both are cut to `most`, which groups that do not overlap never
// pass: offsets that decrease may name all rows for each expert.
template <typename F>
__device__ __forceinline__ int sum_groups(const Grouped& a, int* s_first, int64_t most, F&& of_rows)
{
    __shared__ int64_t s_wave[kWaves];
    int64_t before = 0;
    for (int base = 0; base < a.experts; base += kThreads) {
        const int e = base + (int)threadIdx.x;
        int64_t n = 0;
        if (e < a.experts) {
            int64_t first, end;
            group_range(a, e, first, end);
            n = of_rows((int)(end - first));
        }
        const int64_t to = wave_inclusive_scan(n);
        __syncthreads();
        if (lane_id() == kWave - 1) s_wave[threadIdx.x / kWave] = to;
        __syncthreads();
        int64_t from = before;
        for (int w = 0; w < kWaves; ++w) {
            if (w < (int)threadIdx.x / kWave) from += s_wave[w];
            before += s_wave[w];
        }
        if (e < a.experts) s_first[e] = (int)min(from + to - n, most);
    }
    __syncthreads();
    return uniform((int)min(before, most));
}

// The last group with s_first <= v.
__device__ __forceinline__ int group_at(const int* s_first, int groups, int v)
{
    int e = 0, over = groups;
    while (over - e > 1) {
        const int mid = (e + over) >> 1;
        if (uniform(s_first[mid]) <= v)
            e = mid;
        else
            over = mid;
    }
    return e;
}

// Columns of C; the gradient's C is rows x cols and its depth the group's rows.
template <GroupedOp OP> __device__ __forceinline__ int width_of(const Grouped& a)
{
    return (int)(OP == kProduct ? a.rows : a.cols);
}

// Fills s_first and deals out the tiles. Workgroup i runs on XCD i % 8. A
// product's tiles all cost the same, and each XCD takes an eighth of them. A
// tile of the gradient costs its group's stages and some for its start and end:
// the XCDs' runs end where eighths of that cost do (64 experts whose lengths
// differ by a factor of 8, 65,536 rows in all, 1,536 x 2,048: 589 us with equal
// numbers of tiles, 534 so).
template <GroupedOp OP, int M, int N>
__device__ __forceinline__ Turns deal_tiles(const Grouped& a, int* s_first)
{
    constexpr int kTileCost = 4;  // of a tile beside its stages, in stages
    const int xcd = (int)blockIdx.x % kXcds, among = (int)blockIdx.x / kXcds, per = (int)gridDim.x / kXcds;
    const int wide = (width_of<OP>(a) + N - 1) / N;
    int from, to;
    if constexpr (OP == kGradient) {
        const int each = ((int)a.rows + M - 1) / M * wide;  // tiles of a group
        const int64_t cost = sum_groups(a, s_first, a.m / kDepth + (1 + kTileCost) * (int64_t)a.experts,
                                        [](int rows) { return (rows + kDepth - 1) / kDepth + kTileCost; });
        const auto tile_at = [&](int64_t v) {  // the first tile that starts at v of the cost or behind it
            const int e = group_at(s_first, a.experts, (int)v), first = uniform(s_first[e]);
            const int own = (e + 1 < a.experts ? uniform(s_first[e + 1]) : (int)cost) - first;
            return e * each + (int)(((v - first) * each + own - 1) / own);
        };
        from = xcd == 0 ? 0 : tile_at(cost * xcd / kXcds);
        to = xcd == kXcds - 1 ? a.experts * each : tile_at(cost * (xcd + 1) / kXcds);
    } else {
        const int tiles = sum_groups(a, s_first, a.m / M + a.experts, [](int rows) { return (rows + M - 1) / M; }) * wide;
        const int run = (tiles + kXcds - 1) / kXcds;
        from = xcd * run;
        to = min(from + run, tiles);
    }
    return Turns{from + among, to, per};
}

template <GroupedOp OP, int M, int N>
__device__ __forceinline__ Tile find_tile(const Grouped& a, const Turns& turns, int turn, const int* s_first)
{
    Tile t = {};
    const int tile = turns.at + turn * turns.step;
    t.there = tile < turns.end;
    if (!t.there) return t;
    const int wide = (width_of<OP>(a) + N - 1) / N, block = tile / wide;
    t.n0 = tile % wide * N;
    int in = block;  // the block among the expert's
    if constexpr (OP == kGradient) {
        const int high = ((int)a.rows + M - 1) / M;
        t.e = block / high;
        in = block % high;
    } else {
        t.e = group_at(s_first, a.experts, block);
        in -= uniform(s_first[t.e]);
    }
    int64_t first, end;
    group_range(a, t.e, first, end);
    t.first = uniform((int)first);
    t.end = uniform((int)end);
    t.m0 = OP == kGradient ? in * M : t.first + in * M;
    t.depth = OP == kGradient ? t.end - t.first : (int)a.depth;
    return t;
}

// The rows of x that rows `row[i]` of the tile are; inside the group whatever
// they are, and where the index names none, some row that is there (its products
// are not kept).
template <int N>
__device__ __forceinline__ void group_rows(const Grouped& a, const Tile& t, int (&row)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) row[i] = min(t.m0 + row[i], t.end - 1);
    if (!a.index) return;
#pragma unroll
    for (int i = 0; i < N; ++i) row[i] = a.index[row[i]];
#pragma unroll
    for (int i = 0; i < N; ++i) row[i] = max(row_of_entry(a, row[i]), 0);
}

// 16 bytes a lane straight into LDS, 1 KiB from `to` on. As the compiler's own
// instruction it would make each read of LDS wait for all of these that came
// before, since it cannot tell the ring's slots apart; stage_there() has the waits.
__device__ __forceinline__ void load_to_lds(const char* from, lds_char* to)
{
    const uint32_t at = (uint32_t)(uintptr_t)to;  // uniform
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(from) : "m0");
}

// ---------------------------------------------------------------------------
// Operands that LDS takes directly. Each of a wave's R loads of a stage brings 1
// KiB: 16 rows of 64 bytes along k, or 8 / R lines across it.
// ---------------------------------------------------------------------------
struct Issuer {
    int wave;
    const char* none;  // zeros
    __device__ __forceinline__ Issuer() : wave(uniform((int)threadIdx.x / kWave)), none(reinterpret_cast<const char*>(zeros))
    {
        asm volatile("" : "+s"(wave), "+s"(none));  // not worked out anew at each use
    }
};

template <typename T, int R, bool ACROSS> struct Rows {
    const char* p[R];      // this lane's 16 bytes at k = 0 (across k: of its line)
    int k[ACROSS ? R : 1]; // their k in a stage
    int64_t step;          // bytes from one stage to the next

    // along k: rows `stride` apart; rows_of turns the tile's rows into theirs
    template <typename F>
    __device__ __forceinline__ void begin_along(const T* base, int64_t stride, F&& rows_of)
    {
        const int lane = lane_id(), wave = uniform((int)threadIdx.x / kWave);
        const int seg = (lane % 4) ^ (lane / 8 % 4);  // (row / 2) % 4 = (lane / 8) % 4
        k[0] = seg * 8;
        step = kDepth * (int)sizeof(T);
        int row[R];
#pragma unroll
        for (int i = 0; i < R; ++i) row[i] = (wave * R + i) * 16 + lane / 4;
        rows_of(row);
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = reinterpret_cast<const char*>(base + row[i] * stride + seg * 8);
    }
    // across k: lines `stride` apart from `base` on, of `length` elements
    __device__ __forceinline__ void begin_across(const T* base, int64_t stride, int64_t from, int64_t length)
    {
        const int lane = lane_id(), wave = uniform((int)threadIdx.x / kWave);
        step = kDepth * stride * (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            k[i] = (wave * R + i) * (8 / R) + lane / (8 * R);
            const int64_t at = from + (lane % (8 * R) ^ k[i] % 4 * 2) * 8;
            p[i] = reinterpret_cast<const char*>(base + k[i] * stride + min(at, length - 8));
        }
    }
    // the i-th load of a stage; left: k from its first on, what lies past them is 0
    __device__ __forceinline__ void issue(const Issuer& by, int i, lds_char* stage, int left)
    {
        const char* const from = k[ACROSS ? i : 0] >= left ? by.none : p[i];
        load_to_lds(from, stage + (by.wave * R + i) * 1024);
        p[i] += step;
    }
    // ... 0 in this lane unless `there`
    __device__ __forceinline__ void issue_if(const Issuer& by, int i, lds_char* stage, bool there)
    {
        const char* const from = there ? p[i] : by.none;
        load_to_lds(from, stage + (by.wave * R + i) * 1024);
        p[i] += step;
    }
};

// Lines across k that an index names: a wave's 8 lines of a stage are 8
// successive entries. They are read and turned into addresses in scalar
// registers, a stage ahead, and a lane only chooses between them.
template <typename T, int R> struct IndexedRows {
    static constexpr int W = 8 / R;  // lines of a load
    int first, depth;                // the group's entries, from this wave's first on, and all of them
    int32_t entry[8];
    const char* line[8];             // at the tile's first column; zeros where there is no row
    int most;                        // bytes from there to the last segment that there is
    const char* x;
    __device__ __forceinline__ void begin(const Grouped& g, const Issuer& by, const Tile& t, int from, int length)
    {
        first = t.first + by.wave * 8;
        depth = t.depth - by.wave * 8;
        most = (length - 8 - from) * (int)sizeof(T);
        x = static_cast<const char*>(g.x) + from * (int64_t)sizeof(T);
        fetch(g, 0);
        find(g, by);
    }
    // k0: of the stage
    __device__ __forceinline__ void fetch(const Grouped& g, int k0)
    {
        const auto* const index = (const __attribute__((address_space(4))) int32_t*)g.index + first + k0;
        if (k0 + 8 <= depth) {
#pragma unroll
            for (int i = 0; i < 8; ++i) entry[i] = index[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) entry[i] = k0 + i < depth ? index[i] : -1;
        }
    }
    template <int I> __device__ __forceinline__ void find_one(const Grouped& g, const Issuer& by)
    {
        const uint32_t n = (uint32_t)entry[I], t = (n + __umulhi(n, g.magic)) >> g.shift;
        const char* const at = x + (int64_t)t * (g.x_stride * (int64_t)sizeof(T));
        line[I] = n < g.entries ? at : by.none;
    }
    __device__ __forceinline__ void find(const Grouped& g, const Issuer& by)
    {
        find_one<0>(g, by), find_one<1>(g, by), find_one<2>(g, by), find_one<3>(g, by);
        find_one<4>(g, by), find_one<5>(g, by), find_one<6>(g, by), find_one<7>(g, by);
    }
    // this lane's line of the I-th load
    template <int I> __device__ __forceinline__ const char* choose() const
    {
        const int part = lane_id() / (8 * R);
        const auto pick = [](bool second, const char* a, const char* b) { return second ? b : a; };
        const char* e = pick(part & 1, line[I * W], line[I * W + 1]);
        if constexpr (W >= 4) e = pick(part & 2, e, pick(part & 1, line[I * W + 2], line[I * W + 3]));
        if constexpr (W == 8)
            e = pick(part & 4, e, pick(part & 2, pick(part & 1, line[4], line[5]), pick(part & 1, line[6], line[7])));
        return e;
    }
    template <int I> __device__ __forceinline__ void issue(const Issuer& by, const char* e, lds_char* stage)
    {
        const int lane = lane_id(), k = (by.wave * R + I) * W + lane / (8 * R);
        load_to_lds(e + min((lane % (8 * R) ^ k % 4 * 2) * kVecBytes, most), stage + (by.wave * R + I) * 1024);
    }
};

// One sum. Those of 256 blocks a wave lie in accumulation registers and are moved
// one by one as they are written: left to the compiler they are all moved before
// the first, and what the tiles' loop holds is spilled for it. settle() has to
// come between the last matrix instruction and the first of these.
template <bool MOVED>
__device__ __forceinline__ float sum_of(float acc)
{
    if constexpr (!MOVED) return acc;
    float v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(acc));
    return v;
}
__device__ __forceinline__ void settle()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A wave's part of C: lane l has, of block (j, i), row m = l % 32 and the columns
// n = 8 q + 4 (l / 32) + 0 .. 3 for q = 0 .. 3. `rows`, `cols`: of C from the
// tile on; WHOLE: cols is a multiple of 4.
template <typename G, int TM, int TN, bool WHOLE>
__device__ __forceinline__ void write_tile(const f32x16 (&acc)[TN][TM], G* c, int64_t stride, int rows, int cols, bool add,
                                           uint32_t kept)
{
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    const int m0 = wave / 2 * 32 * TM + lane % 32, n0 = wave % 2 * 32 * TN + lane / 32 * 4;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        if (m0 + 32 * i >= rows) continue;
        G* const row = c + (m0 + 32 * i) * stride + n0;
        const bool keep = kept >> i & 1;
        int left = cols - n0;
        asm volatile("" : "+v"(left));  // compared anew for each row: kept masks would not fit
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = 32 * j + 8 * q;
                if (WHOLE ? n < left : n + 4 <= left) {
                    G g[4];
                    float v[4];
                    if (add) __builtin_memcpy(g, row + n, sizeof(g));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float sum = sum_of<(TM * TN > 4)>(acc[j][i][4 * q + k]);
                        v[k] = keep ? sum : 0.0f;
                        g[k] = (G)(add ? v[k] + (float)g[k] : v[k]);
                    }
                    __builtin_memcpy(row + n, g, sizeof(g));
                } else if (!WHOLE) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (n + k < left) {
                            const float v = keep ? acc[j][i][4 * q + k] : 0.0f;
                            row[n + k] = (G)(add ? v + (float)row[n + k] : v);
                        }
                }
            }
    }
}

template <typename T, typename G, int TM, int TN, GroupedOp OP, bool WHOLE>
__device__ __forceinline__ void write_out(const Grouped& a, const Tile& t, const f32x16 (&acc)[TN][TM])
{
    if constexpr (OP == kGradient) {
        G* const c = static_cast<G*>(a.dw) + ((int64_t)t.e * a.rows + t.m0) * a.cols + t.n0;
        const int rows = (int)a.rows - t.m0, cols = (int)a.cols - t.n0;
        if (WHOLE && t.depth == 0) {  // whole lines of zeros (64 experts of 1,536 x 2,048, 8 of them used: 146 -> 87 us)
            if (a.accumulate) return;
            constexpr int kPer = Vec16<G>::kN, kWide = 64 * TN / kPer;
            for (int i = threadIdx.x; i < 64 * TM * kWide; i += kThreads)
                if (i / kWide < rows && i % kWide * kPer < cols)
                    *reinterpret_cast<typename Vec16<G>::type*>(c + i / kWide * a.cols + i % kWide * kPer) = u32x4{0, 0, 0, 0};
            return;
        }
        if (!a.accumulate)
            write_tile<G, TM, TN, WHOLE>(acc, c, a.cols, rows, cols, false, ~0u);
        else if (t.depth > 0)
            write_tile<G, TM, TN, WHOLE>(acc, c, a.cols, rows, cols, true, ~0u);
    } else {
        uint32_t kept = ~0u;  // bit i: row i of this lane is one that the index names
        if (a.index)
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int r = t.m0 + (int)threadIdx.x / (2 * kWave) * 32 * TM + lane_id() % 32 + 32 * i;
                if (row_of_entry(a, a.index[min(r, t.end - 1)]) < 0) kept &= ~(1u << i);
            }
        write_tile<G, TM, TN, WHOLE>(acc, static_cast<G*>(a.y) + t.m0 * a.y_stride + t.n0, a.y_stride, t.end - t.m0,
                                     width_of<OP>(a) - t.n0, false, kept);
    }
}

// f(0), .. f(N - 1) with each number known to the compiler, so that what it picks stays in registers.
template <typename F, int... I> __device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F&& f)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void for_each(F&& f)
{
    each_of(std::make_integer_sequence<int, N>{}, f);
}

template <typename T, typename G, int TM, int TN, GroupedOp OP, bool INDEXED>
__global__ __launch_bounds__(kThreads, TM * TN > 4 ? 1 : 2) void grouped_kernel(Grouped a)
{
    constexpr int kM = 64 * TM, kN = 64 * TN, kStage = (TM + TN) * kBlockBytes, kLoads = TM + TN;
    __shared__ __align__(128) char ring[kRing * kStage];
    __shared__ int s_first[kMostGroups];
    const Turns turns = deal_tiles<OP, kM, kN>(a, s_first);
    const auto tile_at = [&](int turn) { return find_tile<OP, kM, kN>(a, turns, turn, s_first); };
    Tile now = tile_at(0), ahead = now;
    if (!now.there) return;
    const int lane = lane_id(), wave = uniform((int)threadIdx.x / kWave);
    const int am = wave / 2 * 32 * TM, bn = wave % 2 * 32 * TN;

    const Issuer by;
    // The stream of stages: `ahead` and its k are three stages before what is multiplied.
    Rows<T, TM, OP == kGradient> ra;
    typename std::conditional<INDEXED, IndexedRows<T, TN>, Rows<T, TN, OP != kProduct>>::type rb;
    static_assert(!INDEXED || (OP == kGradient && TM == TN), "the lines of A are those of B");
    int ahead_turn = 0, ahead_k = 0;
    const auto begin = [&] {
        const T* const w = static_cast<const T*>(a.w) + (int64_t)ahead.e * a.rows * a.cols;
        const T* const x = static_cast<const T*>(a.x);
        if constexpr (OP == kGradient) {
            ra.begin_across(static_cast<const T*>(a.y) + ahead.first * a.y_stride, a.y_stride, ahead.m0, a.rows);
            if constexpr (INDEXED)
                rb.begin(a, by, ahead, ahead.n0, a.cols);
            else
                rb.begin_across(x + ahead.first * a.x_stride, a.x_stride, ahead.n0, a.cols);
        } else {
            ra.begin_along(x, a.x_stride, [&](int (&row)[TM]) { group_rows(a, ahead, row); });
            if constexpr (OP == kTransposed)
                rb.begin_across(w, a.cols, ahead.n0, a.cols);
            else
                rb.begin_along(w, a.cols, [&](int (&row)[TN]) {
#pragma unroll
                    for (int i = 0; i < TN; ++i) row[i] = min(ahead.n0 + row[i], (int)a.rows - 1);
                });
        }
    };
    const char* chosen[TN];  // this lane's lines of x
    const auto issue_a = [&](auto step, lds_char* stage, int left) {
        constexpr int i = decltype(step)::value;
        if constexpr (INDEXED) {  // a row of padding is left out, whatever dy has there
            chosen[i] = rb.template choose<i>();
            ra.issue_if(by, i, stage, chosen[i] != by.none);
        } else {
            ra.issue(by, i, stage, left);
        }
    };
    const auto issue = [&](auto step, int slot) {  // one of kLoads of a stage
        constexpr int i = decltype(step)::value;
        lds_char* const stage = (lds_char*)(ring + slot * kStage);
        const int left = ahead.depth - ahead_k;
        if constexpr (i < TM)
            issue_a(step, stage, left);
        else if constexpr (INDEXED)
            rb.template issue<i - TM>(by, chosen[i - TM], stage + TM * kBlockBytes);
        else
            rb.issue(by, i - TM, stage + TM * kBlockBytes, left);
    };
    const auto next = [&] {  // once the tile's last stage is on its way
        if (ahead_k < ahead.depth || !ahead.there) return;
        ahead = tile_at(++ahead_turn);  // none left: depth 0, zeros
        ahead_k = 0;
        if (ahead.there)
            begin();
        else if constexpr (INDEXED)
            rb.depth = 0;  // no entry of the last group again
    };
    u32x4 fa[2][TM], fb[2][TN];
    const auto read = [&](auto step, int slot, auto half) {  // one of kLoads fragments
        constexpr int i = decltype(step)::value, kk = decltype(half)::value;
        const lds_char* const stage = (const lds_char*)(ring + slot * kStage);
        if constexpr (i < TM)
            fa[kk][i] = read_fragment<TM, OP == kGradient>(stage, am, i, kk, lane);
        else
            fb[kk][i - TM] = read_fragment<TN, OP != kProduct>(stage + TM * kBlockBytes, bn, i - TM, kk, lane);
    };
    constexpr std::integral_constant<int, 0> kFirst;
    constexpr std::integral_constant<int, 1> kSecond;
    f32x16 acc[TN][TM];
    // The products of a half, and between them, each in its place, `count` other steps.
    const auto multiply = [&](auto half, auto count, auto&& step) {
        constexpr int kk = decltype(half)::value, kSteps = decltype(count)::value;
        constexpr int kEach = (kSteps + TM * TN - 1) / (TM * TN);
        __builtin_amdgcn_sched_barrier(0);
        for_each<TM * TN>([&](auto at) {
            constexpr int t = decltype(at)::value, j = t / TM, i = t % TM;
            acc[j][i] = mma32<T>(fb[kk][j], fa[kk][i], acc[j][i]);
            for_each<kEach>([&](auto s) {
                constexpr int n = t * kEach + decltype(s)::value;
                if constexpr (n < kSteps) step(std::integral_constant<int, n>{});
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // At most the two stages after the next are still to come; this wave's reads
    // are done, so that after the barrier the slot they were of may be filled.
    const auto stage_there = [&] {
        if constexpr (kLoads == 8)
            asm volatile("s_waitcnt vmcnt(16) lgkmcnt(0)" ::: "memory");
        else if constexpr (kLoads == 4)
            asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)" ::: "memory");
        else
            asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    static_assert(kLoads == 8 || kLoads == 4 || kLoads == 2, "the waits above");

    begin();
    for (int slot = 0; slot < kRing - 1; ++slot) {
        for_each<kLoads>([&](auto i) { issue(i, slot); });
        ahead_k += kDepth;
        if constexpr (INDEXED) {
            rb.fetch(a, ahead_k);
            rb.find(a, by);
        }
        next();
    }
    stage_there();
    for_each<kLoads>([&](auto i) { read(i, 0, kFirst); });
    int slot = 0, turn = 0;
    for (;;) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int k = 0; k < 16; ++k) acc[j][i][k] = 0.0f;
        for (int k0 = 0; k0 < now.depth || k0 == 0; k0 += kDepth) {
            const int free = (slot + kRing - 1) % kRing;
            if constexpr (INDEXED) rb.fetch(a, ahead_k + kDepth);
            multiply(kFirst, std::integral_constant<int, 2 * kLoads>{}, [&](auto i) {
                if constexpr (decltype(i)::value < kLoads)
                    read(i, slot, kSecond);
                else
                    issue(std::integral_constant<int, decltype(i)::value - kLoads>{}, free);
            });
            ahead_k += kDepth;
            stage_there();
            slot = (slot + 1) % kRing;
            multiply(kSecond, std::integral_constant<int, kLoads + (INDEXED ? 8 : 0)>{}, [&](auto i) {
                if constexpr (decltype(i)::value < kLoads)
                    read(i, slot, kFirst);
                else if constexpr (INDEXED)
                    rb.template find_one<decltype(i)::value - kLoads>(a, by);
            });
            next();
        }
        settle();
        write_out<T, G, TM, TN, OP, true>(a, now, acc);
        now = tile_at(++turn);
        if (!now.there) break;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the workgroup
}

// ---------------------------------------------------------------------------
// Operands of any alignment and length, through registers, kAhead stages ahead
// (1,003 tokens, top-2 of 20, 777 x 1,000 transposed in fp16: 41 us one stage
// ahead, 23 so).
// ---------------------------------------------------------------------------
constexpr int kAhead = 4;

template <typename T, int R, bool ACROSS> struct RowsOdd {
    int64_t from, length;  // across k: the tile's first element of a line, and a line's elements
    u32x4 staged[kAhead][R];
    uint32_t there[kAhead];  // bit i: piece i is of a line that there is
    static __device__ __forceinline__ int place(int i) { return ACROSS ? (i * kThreads + (int)threadIdx.x) / (8 * R) : i * 64 + (int)threadIdx.x / 4; }
    static __device__ __forceinline__ int segment(int i) { return ACROSS ? (i * kThreads + (int)threadIdx.x) % (8 * R) : (int)threadIdx.x % 4; }
    __device__ __forceinline__ int64_t element(int i, int k0) const { return (ACROSS ? from : k0) + segment(i) * 8; }
    // line_of(place, &there): a line that is there in any case. A piece that ends
    // past its line is loaded from the line's last 16 bytes, and moved down only
    // as it is put into LDS (zeros unless `keep`), so that loading waits for nothing.
    template <typename F>
    __device__ __forceinline__ void load(int set, int k0, int depth, F&& line_of)
    {
        const int64_t all = ACROSS ? length : depth;
        there[set] = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            bool is = true;
            const T* const l = line_of(place(i), is);
            there[set] |= (uint32_t)is << i;
            const int64_t at = element(i, k0);
            if (all >= 8)  // uniform
                staged[set][i] = *reinterpret_cast<const typename Vec16<T>::type*>(l + min(at, all - 8));
            else
                staged[set][i] = at < all ? load_end<T>(l, at, all) : u32x4{0, 0, 0, 0};
        }
    }
    __device__ __forceinline__ void put(int set, int k0, int depth, lds_char* stage, bool keep = true) const
    {
        const int64_t all = ACROSS ? length : depth;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int p = place(i), s = segment(i);
            const int64_t at = element(i, k0);
            u32x4 v = staged[set][i];
            if (all >= 8 && at > all - 8) v = move_down<T>(v, at - (all - 8));
            if (!keep || !(there[set] >> i & 1)) v = u32x4{0, 0, 0, 0};
            lds_char* const to = ACROSS ? stage + p * (128 * R) + (s ^ p % 4 * 2) * 16 : stage + p * 64 + ((s ^ (p >> 1)) & 3) * 16;
            *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(to) = v;
        }
    }
};

template <typename T, typename G, int TM, int TN, GroupedOp OP>
__global__ __launch_bounds__(kThreads, 2) void grouped_odd_kernel(Grouped a)
{
    constexpr int kM = 64 * TM, kN = 64 * TN, kStage = (TM + TN) * kBlockBytes;
    __shared__ __align__(128) char ring[2 * kStage];
    __shared__ int s_first[kMostGroups];
    const Turns turns = deal_tiles<OP, kM, kN>(a, s_first);
    const int lane = lane_id(), wave = uniform((int)threadIdx.x / kWave);
    const int am = wave / 2 * 32 * TM, bn = wave % 2 * 32 * TN;
    const T* const x = static_cast<const T*>(a.x);
    for (int turn = 0;; ++turn) {
        const Tile t = find_tile<OP, kM, kN>(a, turns, turn, s_first);
        if (!t.there) break;
        const T* const w = static_cast<const T*>(a.w) + (int64_t)t.e * a.rows * a.cols;
        RowsOdd<T, TM, OP == kGradient> ra;
        RowsOdd<T, TN, OP != kProduct> rb;
        ra.from = t.m0;
        ra.length = a.rows;
        rb.from = t.n0;
        rb.length = a.cols;
        int xrow[TM];  // of the rows that this thread loads
        if constexpr (OP != kGradient) {
#pragma unroll
            for (int i = 0; i < TM; ++i) xrow[i] = RowsOdd<T, TM, false>::place(i);
            group_rows(a, t, xrow);
        }
        static_assert(OP != kGradient || TM == 1, "one entry of the index for what a thread loads of dy");
        int32_t entry[kAhead];  // of the row of dy
        const auto load = [&](int set, int k0) {
            if constexpr (OP == kGradient) {
                ra.load(set, k0, t.depth, [&](int k, bool& is) {
                    const int r = t.first + min(k0 + k, t.depth - 1);
                    is = k0 + k < t.depth;
                    entry[set] = a.index ? a.index[r] : 0;
                    return static_cast<const T*>(a.y) + r * a.y_stride;
                });
                rb.load(set, k0, t.depth, [&](int k, bool& is) {
                    const int64_t r = batch_row(a, t.first + min(k0 + k, t.depth - 1));
                    is = k0 + k < t.depth && r >= 0;
                    return x + max(r, (int64_t)0) * a.x_stride;
                });
            } else {
                int i = 0;
                ra.load(set, k0, t.depth, [&](int, bool&) { return x + xrow[i++] * a.x_stride; });
                if constexpr (OP == kTransposed)
                    rb.load(set, k0, t.depth, [&](int k, bool& is) {
                        is = k0 + k < t.depth;
                        return w + (int64_t)min(k0 + k, t.depth - 1) * a.cols;
                    });
                else
                    rb.load(set, k0, t.depth, [&](int n, bool&) { return w + min((int64_t)t.n0 + n, a.rows - 1) * a.cols; });
            }
        };
        f32x16 acc[TN][TM] = {};
        const int stages = (t.depth + kDepth - 1) / kDepth;
        __syncthreads();  // the tile before is done with the slots
        for_each<kAhead>([&](auto u) {
            constexpr int set = decltype(u)::value;
            if (set < stages) load(set, set * kDepth);
        });
        for (int s0 = 0; s0 < stages; s0 += kAhead)
            for_each<kAhead>([&](auto u) {
                constexpr int set = decltype(u)::value;
                const int s = s0 + set;
                if (s >= stages) return;  // uniform
                lds_char* const stage = (lds_char*)(ring + set % 2 * kStage);
                bool keep = true;  // a row of padding is left out, whatever dy has there
                if constexpr (OP == kGradient) keep = !a.index || row_of_entry(a, entry[set]) >= 0;
                ra.put(set, s * kDepth, t.depth, stage, keep);  // all are done with the slot: two stages ago it was read, one ago there was a barrier
                rb.put(set, s * kDepth, t.depth, stage + TM * kBlockBytes);
                if (s + kAhead < stages) load(set, (s + kAhead) * kDepth);
                __syncthreads();
                for_each<2>([&](auto half) {
                    constexpr int kk = decltype(half)::value;
                    u32x4 fa[TM], fb[TN];
#pragma unroll
                    for (int i = 0; i < TM; ++i) fa[i] = read_fragment<TM, OP == kGradient>(stage, am, i, kk, lane);
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        fb[j] = read_fragment<TN, OP != kProduct>(stage + TM * kBlockBytes, bn, j, kk, lane);
#pragma unroll
                    for (int j = 0; j < TN; ++j)
#pragma unroll
                        for (int i = 0; i < TM; ++i) acc[j][i] = mma32<T>(fb[j], fa[i], acc[j][i]);
                });
            });
        write_out<T, G, TM, TN, OP, false>(a, t, acc);
    }
}

int grouped_most_experts() { return kMostGroups; }

constexpr int kCus = 256;

// Tiles of C in tiles of m x n, at most (a product's go by the lengths of the groups).
static int64_t most_tiles(GroupedOp op, const Grouped& a, int m, int n)
{
    const int64_t wide = ((op == kProduct ? a.rows : a.cols) + n - 1) / n;
    if (op == kGradient) return a.experts * ((a.rows + m - 1) / m) * wide;
    return ((a.m + m - 1) / m + (a.experts < a.m ? a.experts : a.m)) * wide;
}

int64_t grouped_tiles(const Grouped& a, bool gradient)
{
    return most_tiles(gradient ? kGradient : a.transposed ? kTransposed : kProduct, a, 64, 64);
}

static dim3 resident(int64_t tiles, int per_cu)
{
    const int64_t most = (int64_t)kCus * per_cu, need = (tiles + kXcds - 1) / kXcds * kXcds;
    return dim3((unsigned)(need < most ? need : most));
}

template <typename T, typename G, GroupedOp OP> static void launch_op(const Grouped& a, hipStream_t stream)
{
    const auto even = [](const void* p, int64_t stride) { return (uintptr_t)p % 16 == 0 && stride % 8 == 0; };
    const dim3 block(kThreads);
    const bool whole = a.rows % 8 == 0 && a.cols % 8 == 0 && a.x_rows > 0 && even(a.x, a.x_stride) &&
                       (OP == kGradient ? even(a.y, a.y_stride) : even(a.w, 0) && a.depth > 0);
    if (!whole) {
        grouped_odd_kernel<T, G, 1, 2, OP><<<resident(most_tiles(OP, a, 64, 128), 2), block, 0, stream>>>(a);
        return;
    }
    const auto go = [&](auto tm, auto indexed) {
        constexpr int R = decltype(tm)::value;
        const dim3 grid = resident(most_tiles(OP, a, 64 * R, 64 * R), R == 4 ? 1 : R == 2 ? 2 : 4);
        grouped_kernel<T, G, R, R, OP, decltype(indexed)::value><<<grid, block, 0, stream>>>(a);
    };
    // Tiles of 256 where there are enough of them: two for each CU in a product
    // (65,536 rows of 64 experts, 1,536 x 2,048: 449 us against 613 with tiles of
    // 128; at 544 tiles 103 and 105, at 384 tiles 64 and 55), four in a gradient
    // whose groups have 512 rows on average (that gradient: 518 and 744 us; 512
    // tiles 74 and 58; 1,024 tiles of 128 rows 81 and 69). Tiles of 128 down to half
    // a tile for each CU in a product (192 tiles 14.2 us, with tiles of 64 16.9; 108
    // tiles 18.8 and 14.6), a tile in a gradient (512: 17.5 and 20.7; 64: 42 and 27).
    // All of a product's were timed with hundreds of rows to a group; how many rows a
    // group has is not asked, and short groups are padded to the tile.
    const auto sized = [&](auto indexed) {
        const int64_t large = most_tiles(OP, a, 256, 256), medium = most_tiles(OP, a, 128, 128);
        const bool deep = OP != kGradient || a.m / 512 >= a.experts;
        if (deep && large >= (OP == kGradient ? 4 : 2) * kCus)
            go(std::integral_constant<int, 4>{}, indexed);
        else if (medium >= (OP == kGradient ? kCus : kCus / 2))
            go(std::integral_constant<int, 2>{}, indexed);
        else
            go(std::integral_constant<int, 1>{}, indexed);
    };
    if constexpr (OP == kGradient) {
        if (a.index) {
            sized(std::true_type{});
            return;
        }
    }
    sized(std::false_type{});
}

template <typename T> static void launch_product(const Grouped& a, hipStream_t stream)
{
    if (a.transposed)
        launch_op<T, T, kTransposed>(a, stream);
    else
        launch_op<T, T, kProduct>(a, stream);
}

hipError_t launch_grouped_matmul(ElemKind kind, const Grouped& a, hipStream_t stream)
{
    if (kind == kBF16)
        launch_product<bf16>(a, stream);
    else
        launch_product<fp16>(a, stream);
    return hipGetLastError();
}

hipError_t launch_grouped_matmul_grad(ElemKind kind, ElemKind grad_kind, const Grouped& a, hipStream_t stream)
{
    if (kind == kBF16) {
        if (grad_kind == kF32)
            launch_op<bf16, float, kGradient>(a, stream);
        else
            launch_op<bf16, bf16, kGradient>(a, stream);
    } else {
        if (grad_kind == kF32)
            launch_op<fp16, float, kGradient>(a, stream);
        else
            launch_op<fp16, fp16, kGradient>(a, stream);
    }
    return hipGetLastError();
}

}  // namespace ds
