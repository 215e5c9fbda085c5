// moe_experts.hip -- the experts of a mixture-of-experts layer for a few
// tokens: for every token t and choice j with expert e = ids[t, j],
//
//   h = silu(G_e x_t) * (U_e x_t)          G_e, U_e: the first and the last F rows of w_in[e]
//   y_t = sum over j of weights[t, j] * (w_out[e] h)
//
// With a few tokens the weights are what has to be read (3 D F values per
// expert that any token chose, once), so the kernels are built to stream
// them: weights go from memory straight into the A operand of the matrix
// instructions, 16 rows to a tile, and the expert's tokens, at most 16 to a
// column block, are the B operand, read from the cache.
//
// Three launches: gate/up products and activation into `h` (one row per
// assignment, in x's type), down products into `part` (one 32-bit row per
// assignment), and the weighted sum over each token's choices, in order of
// the choices, so that the result is the same on every run. There is no
// alignment launch before them: each workgroup finds its expert and that
// expert's assignments in the ids itself.
#include "device_scan.hpp"
#include "float_types.hpp"
#include "launch.hpp"

namespace ds {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Operands of one matrix instruction (16 x 16 outputs, 32 deep): 8 values per lane.
template <typename X> struct Frag;
template <> struct Frag<bf16> {
    typedef bf16x8 type;
    static __device__ __forceinline__ f32x4 mma(type a, type b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Frag<fp16> {
    typedef f16x8 type;
    static __device__ __forceinline__ f32x4 mma(type a, type b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// Eight e4m3 values as X (exact: both 16-bit types hold every one of them).
template <typename X>
__device__ __forceinline__ typename Frag<X>::type widen8(uint32_t lo, uint32_t hi)
{
    union {
        typename Frag<X>::type v;
        uint32_t u[4];
    } r;
    if constexpr (sizeof(X) == 2 && __is_same(X, bf16)) {
        r.u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
        r.u[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
        r.u[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
        r.u[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
    } else {
        r.u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
        r.u[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
        r.u[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
        r.u[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
    }
    return r.v;
}

// A step covers 64 of the depth: lane l of a wave holds row (A) or token (B)
// l % 16, depth (l / 16) * 16 .. + 15 of the step, as two fragments of 8. Both
// operands use this order, so the products pair up; a row's 128 bytes (64 in
// 8 bits) are then read by four lanes side by side.
constexpr int kStep = 64;
constexpr int kLaneDepth = 16;

// One lane's 16 values of a step, as loaded (16-bit types: two 16-byte
// vectors; 8-bit: one).
template <typename W> struct StepRegs {
    u32x4 v[kLaneDepth * sizeof(W) / 16];
};

template <typename W>
__device__ __forceinline__ StepRegs<W> load_step(const W* __restrict__ p)
{
    StepRegs<W> r;
    constexpr int kN = kLaneDepth * sizeof(W) / 16;
    const typename Vec16<W>::type* q = reinterpret_cast<const typename Vec16<W>::type*>(p);
#pragma unroll
    for (int i = 0; i < kN; ++i) r.v[i] = q[i];
    return r;
}

// The same for the step at the end of the depth: values past `valid` are 0.
template <typename W>
__device__ __forceinline__ StepRegs<W> load_step_tail(const W* __restrict__ p, int valid)
{
    union {
        StepRegs<W> r;
        W w[kLaneDepth];
    } u;
    __builtin_memset(&u, 0, sizeof(u));
#pragma unroll
    for (int i = 0; i < kLaneDepth; ++i)
        if (i < valid) u.w[i] = p[i];
    return u.r;
}

template <typename X, typename W>
__device__ __forceinline__ typename Frag<X>::type fragment(const StepRegs<W>& r, int half)
{
    if constexpr (sizeof(W) == 1)
        return widen8<X>(r.v[0][half * 2], r.v[0][half * 2 + 1]);
    else
        return __builtin_bit_cast(typename Frag<X>::type, r.v[half]);
}

// Products of two 16-row tiles with TT blocks of 16 tokens, over the depth
// [k0, k1): acc[tile][block]. `rows`: this lane's row of each tile; `tok`:
// this lane's token row of each block. k0 is a multiple of 128; `scale`:
// null, or this lane's scales, for its four output rows of each tile, of the
// first block of 128 of the depth; the next block's are one element on.
template <typename X, typename W, int TT>
__device__ __forceinline__ void product(const W* const (&rows)[2], const X* const (&tok)[TT],
                                        const float* const (&scale)[2][4], int k0, int k1, int lane,
                                        f32x4 (&acc)[2][TT])
{
    const int off = lane / 16 * kLaneDepth;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int b = 0; b < TT; ++b) acc[r][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int kBlock = 2 * kStep;  // 128 deep
    for (int k = k0; k < k1; k += kBlock) {
        f32x4 sum[2][TT];
        if constexpr (sizeof(W) == 1) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int b = 0; b < TT; ++b) sum[r][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        StepRegs<W> a[2][2];
        StepRegs<X> x[2][TT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int at = k + s * kStep + off, valid = k1 - at;
            if (k + (s + 1) * kStep <= k1) {  // uniform
#pragma unroll
                for (int r = 0; r < 2; ++r) a[s][r] = load_step<W>(rows[r] + at);
#pragma unroll
                for (int b = 0; b < TT; ++b) x[s][b] = load_step<X>(tok[b] + at);
            } else {
#pragma unroll
                for (int r = 0; r < 2; ++r) a[s][r] = load_step_tail<W>(rows[r] + at, valid);
#pragma unroll
                for (int b = 0; b < TT; ++b) x[s][b] = load_step_tail<X>(tok[b] + at, valid);
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const typename Frag<X>::type af = fragment<X, W>(a[s][r], half);
#pragma unroll
                    for (int b = 0; b < TT; ++b) {
                        const typename Frag<X>::type bf = fragment<X, X>(x[s][b], half);
                        if constexpr (sizeof(W) == 1)
                            sum[r][b] = Frag<X>::mma(af, bf, sum[r][b]);
                        else
                            acc[r][b] = Frag<X>::mma(af, bf, acc[r][b]);
                    }
                }
        if constexpr (sizeof(W) == 1) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                f32x4 sc;
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[i] = scale[r][i][(k - k0) / kBlock];
#pragma unroll
                for (int b = 0; b < TT; ++b) acc[r][b] += sc * sum[r][b];
            }
        }
    }
}

// Which expert a workgroup serves, and that expert's assignments, found in
// the ids by the workgroup itself. With at least as many slots as experts,
// slot s is expert s; with fewer (few assignments), slot s is the s-th expert
// that any assignment names.
struct Found {
    int expert, count;  // count 0: nothing to do
};

__device__ __forceinline__ Found find_assignments(const int32_t* __restrict__ ids, int n, int experts, int slots,
                                                  int slot, uint16_t* list)
{
    __shared__ uint32_t s_used[kThreads];  // bit e: expert e is named (8,192 experts at most)
    __shared__ int s_expert, s_count;
    if (threadIdx.x == 0) {
        s_expert = slots >= experts ? slot : -1;
        s_count = 0;
    }
    if (slots < experts) {
        s_used[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int e = ids[i];
            if (e >= 0 && e < experts) atomicOr(&s_used[e / 32], 1u << (e % 32));
        }
        __syncthreads();
        if (threadIdx.x < kWave) {
            // lane l counts words 4 l .. 4 l + 3; the lane that holds the slot-th set bit walks its words
            uint32_t w[4], own = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = s_used[threadIdx.x * 4 + j];
                own += (uint32_t)__builtin_popcount(w[j]);
            }
            const uint32_t before = wave_inclusive_scan(own) - own;
            if ((uint32_t)slot >= before && (uint32_t)slot < before + own) {
                int left = slot - (int)before;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t bits = w[j];
                    while (bits) {
                        if (left-- == 0) s_expert = ((int)threadIdx.x * 4 + j) * 32 + __builtin_ctz(bits);
                        bits &= bits - 1;
                    }
                }
            }
        }
    }
    __syncthreads();
    const int expert = s_expert;
    if (expert >= 0) {
        for (int i = threadIdx.x; i < n; i += kThreads)
            if (ids[i] == expert) list[atomicAdd(&s_count, 1)] = (uint16_t)i;
    }
    __syncthreads();
    return Found{expert, expert >= 0 ? s_count : 0};
}

struct ExpertArgs {
    const int32_t* ids;
    const void *x, *w, *scale;  // scale: [experts][ceil(rows / 128)][ceil(depth / 128)], or null
    void* out;
    int64_t x_stride;  // elements between rows of x
    int n, top_k, experts, slots, slices;
    int rows, depth;   // of one expert's matrix; gate/up: rows = F (of 2 F), depth = D; down: rows = D, depth = F
};

// GATED: tiles are gate rows and the up rows that go with them, x rows are the
// tokens', the output is silu(gate) * up, in X. Otherwise: two tiles of
// neighbouring rows, x rows are the assignments', the output is 32-bit sums.
// PARTS waves share a pair of tiles, each with a part of the depth; a
// workgroup has 4 / PARTS pairs.
template <typename X, typename W, int TT, bool GATED, int PARTS>
__device__ __forceinline__ void expert_block(const ExpertArgs& a, int expert, const uint16_t* list, int first,
                                             int count, int slice, f32x4* s_part)
{
    constexpr int kPairs = kWaves / PARTS;
    const int lane = lane_id(), wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int part = wave % PARTS, pair = slice * kPairs + wave / PARTS;
    const int row0 = pair * (GATED ? 16 : 32);
    const int64_t all_rows = GATED ? 2 * (int64_t)a.rows : a.rows;
    const W* w = (const W*)a.w + (int64_t)expert * all_rows * a.depth;
    const int grid_cols = (a.depth + 127) / 128, grid_rows = (int)((all_rows + 127) / 128);
    // the part of the depth, in whole blocks of 128
    const int blocks = grid_cols, each = (blocks + PARTS - 1) / PARTS;
    const int k0 = part * each * 128, k1 = min((part + 1) * each * 128, a.depth);
    const W* rows[2];
    const float* scale[2][4];
    int64_t tile_row[2];  // first row of each tile in the expert's matrix
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        tile_row[r] = GATED ? (int64_t)r * a.rows + row0 : row0 + 16 * r;
        const int64_t end = GATED ? (int64_t)(r + 1) * a.rows : a.rows;
        const int64_t mine = tile_row[r] + lane % 16;
        rows[r] = w + (mine < end ? mine : end - 1) * a.depth;  // rows past the end repeat the last one
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            scale[r][i] = nullptr;
            if constexpr (sizeof(W) == 1) {
                const int64_t out_row = tile_row[r] + lane / 16 * 4 + i;
                scale[r][i] = (const float*)a.scale +
                              ((int64_t)expert * grid_rows + (out_row < end ? out_row : end - 1) / 128) * grid_cols +
                              k0 / 128;
            }
        }
    }
    const X* tok[TT];
    int assign[TT];
#pragma unroll
    for (int b = 0; b < TT; ++b) {
        const int at = first + b * 16 + lane % 16;
        assign[b] = list[at < count ? at : count - 1];  // columns past the end repeat the last one
        tok[b] = (const X*)a.x + (int64_t)(GATED ? assign[b] / a.top_k : assign[b]) * a.x_stride;
        if (at >= count) assign[b] = -1;
    }
    f32x4 acc[2][TT];
    if (row0 < a.rows && k0 < k1) {
        product<X, W, TT>(rows, tok, scale, k0, k1, lane, acc);
    } else {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < TT; ++b) acc[r][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if constexpr (PARTS > 1) {  // PARTS == kWaves: one pair per workgroup
        static_assert(PARTS == kWaves, "the parts of one pair are the workgroup's waves");
        __syncthreads();  // the previous block's sums have been read
        if (wave > 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int b = 0; b < TT; ++b) s_part[((wave - 1) * 2 * TT + r * TT + b) * kWave + lane] = acc[r][b];
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int p = 0; p < PARTS - 1; ++p)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int b = 0; b < TT; ++b) acc[r][b] += s_part[(p * 2 * TT + r * TT + b) * kWave + lane];
    }
    if (row0 >= a.rows) return;
    // lane l holds output rows (l / 16) * 4 .. + 3 of each tile for token l % 16 of each block
    const int r0 = lane / 16 * 4;
#pragma unroll
    for (int b = 0; b < TT; ++b) {
        if (assign[b] < 0) continue;
        if constexpr (GATED) {
            X* out = (X*)a.out + (int64_t)assign[b] * a.rows + row0 + r0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g = acc[0][b][i], u = acc[1][b][i];
                if (row0 + r0 + i < a.rows) out[i] = (X)(g / (1.0f + expf(-g)) * u);
            }
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float* out = (float*)a.out + (int64_t)assign[b] * a.rows + row0 + 16 * r + r0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (row0 + 16 * r + r0 + i < a.rows) out[i] = acc[r][b][i];
            }
        }
    }
}

constexpr int kMostBlocks = 4;  // blocks of 16 tokens that a wave holds at once

template <typename X, typename W, bool GATED, int PARTS>
__global__ __launch_bounds__(kThreads) void expert_kernel(ExpertArgs a)
{
    extern __shared__ __align__(16) char s_mem[];
    f32x4* s_part = reinterpret_cast<f32x4*>(s_mem);
    uint16_t* list = reinterpret_cast<uint16_t*>(
        s_mem + (PARTS > 1 ? (PARTS - 1) * 2 * kMostBlocks * kWave * sizeof(f32x4) : 0));
    const int slot = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
    const Found f = find_assignments(a.ids, a.n, a.experts, a.slots, slot, list);
    int first = 0;
    while (f.count - first > 32) {
        expert_block<X, W, 4, GATED, PARTS>(a, f.expert, list, first, f.count, slice, s_part);
        first += 64;
    }
    if (f.count - first > 16)
        expert_block<X, W, 2, GATED, PARTS>(a, f.expert, list, first, f.count, slice, s_part);
    else if (f.count - first > 0)
        expert_block<X, W, 1, GATED, PARTS>(a, f.expert, list, first, f.count, slice, s_part);
}

// y_t = sum over j of weights[t, j] * part[t, j], choices outside the experts left out.
template <typename X>
__global__ __launch_bounds__(kThreads) void expert_sum_kernel(const float* __restrict__ part,
                                                              const int32_t* __restrict__ ids,
                                                              const float* __restrict__ weights, int tokens, int top_k,
                                                              int experts, int dim, X* __restrict__ y,
                                                              int64_t y_stride)
{
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int t = (int)(at / dim), d = (int)(at % dim);
    if (t >= tokens) return;
    float sum = 0.0f;
    for (int j = 0; j < top_k; ++j) {
        const int e = ids[t * top_k + j];
        if (e >= 0 && e < experts) sum += weights[t * top_k + j] * part[((int64_t)t * top_k + j) * dim + d];
    }
    y[t * y_stride + d] = (X)sum;
}

int64_t experts_max_assignments() { return 8192; }
int experts_max_experts() { return kThreads * 32; }

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t experts_h_bytes(int64_t n, int hidden) { return ceil_div(n * hidden * 2, 256) * 256; }
int64_t experts_aux_bytes(int64_t n, int dim, int hidden) { return experts_h_bytes(n, hidden) + n * dim * 4; }

template <typename X, typename W, bool GATED>
static hipError_t launch_expert_kernel(ExpertArgs a, hipStream_t stream)
{
    // A wave streams a whole pair of tiles where that gives every CU work;
    // with few experts the four waves of a workgroup share one pair.
    const int64_t pairs = ceil_div(a.rows, GATED ? 16 : 32);
    const bool whole = a.slots * ceil_div(pairs, kWaves) >= 1024;
    a.slices = (int)(whole ? ceil_div(pairs, kWaves) : pairs);
    const dim3 grid((unsigned)((int64_t)a.slots * a.slices)), block(kThreads);
    const size_t list = (size_t)((a.n + 7) / 8 * 8) * sizeof(uint16_t);
    if (whole)
        expert_kernel<X, W, GATED, 1><<<grid, block, list, stream>>>(a);
    else
        expert_kernel<X, W, GATED, kWaves>
            <<<grid, block, list + (kWaves - 1) * 2 * kMostBlocks * kWave * sizeof(f32x4), stream>>>(a);
    return hipGetLastError();
}

template <typename X, typename W>
static hipError_t experts_typed(const ExpertsCall& c, char* aux, hipStream_t stream)
{
    const int n = (int)(c.tokens * c.top_k);
    char *h = aux, *part = aux + experts_h_bytes(n, c.hidden);
    const int slots = c.experts < n ? c.experts : n;
    ExpertArgs a{c.ids, c.x, c.w_in, c.w_in_scale, h, c.x_stride, n, c.top_k, c.experts, slots, 0, c.hidden, c.dim};
    hipError_t e = launch_expert_kernel<X, W, true>(a, stream);
    if (e != hipSuccess) return e;
    ExpertArgs b{c.ids, h, c.w_out, c.w_out_scale, part, c.hidden, n, c.top_k, c.experts, slots, 0, c.dim, c.hidden};
    e = launch_expert_kernel<X, W, false>(b, stream);
    if (e != hipSuccess) return e;
    const int64_t items = (int64_t)c.tokens * c.dim;
    expert_sum_kernel<X><<<dim3((unsigned)ceil_div(items, kThreads)), dim3(kThreads), 0, stream>>>(
        (const float*)part, c.ids, c.weights, (int)c.tokens, c.top_k, c.experts, c.dim, (X*)c.y, c.y_stride);
    return hipGetLastError();
}

hipError_t launch_moe_experts(ElemKind kind, bool eight_bit, const ExpertsCall& c, char* aux, hipStream_t stream)
{
    if (kind == kBF16)
        return eight_bit ? experts_typed<bf16, fp8>(c, aux, stream) : experts_typed<bf16, bf16>(c, aux, stream);
    if (kind == kF16)
        return eight_bit ? experts_typed<fp16, fp8>(c, aux, stream) : experts_typed<fp16, fp16>(c, aux, stream);
    return hipErrorInvalidValue;
}

}  // namespace ds
