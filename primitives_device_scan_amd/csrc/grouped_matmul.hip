// grouped_matmul.hip -- matrix products grouped by expert: rows [offsets[e],
// offsets[e + 1]) of a batch belong to expert e,
//
//   y_r = W_e x_r   or, transposed, y_r = W_e^T x_r          W_e: rows x cols
//   dW_e = sum over its rows r of dy_r x_r^T
//
// Row r of the batch is row r of x, or, with an index, row index[r] / top_k of
// it (zeros where that is no row): the batch that the MoE alignment orders.
#include "float_types.hpp"
#include "launch.hpp"

namespace ds {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(f16x8 a, f16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
template <typename T> struct Vec8;
template <> struct Vec8<bf16> { using type = bf16x8; };
template <> struct Vec8<fp16> { using type = f16x8; };

__device__ __forceinline__ void group_range(const Grouped& a, int e, int64_t& first, int64_t& end)
{
    first = min(max((int64_t)a.offsets[e], (int64_t)0), a.m);
    end = min(max((int64_t)a.offsets[e + 1], first), a.m);
}

// The row of x that row r of the batch is, or -1.
__device__ __forceinline__ int64_t batch_row(const Grouped& a, int64_t r)
{
    if (!a.index) return r;
    const int64_t i = a.index[r];
    const int64_t t = i / a.top_k;
    return i >= 0 && t < a.x_rows ? t : -1;
}

constexpr int kTile = 64, kDepth = 32, kPad = 8;

// C (64 x 64) of a workgroup's four waves, each a 32 x 32 quarter.
template <typename T, typename LA, typename LB, typename ST>
__device__ __forceinline__ void tile_product(int64_t depth, LA&& load_a, LB&& load_b, ST&& store)
{
    __shared__ T sa[kTile][kDepth + kPad], sb[kTile][kDepth + kPad];
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    f32x4 acc[2][2] = {};
    for (int64_t k0 = 0; k0 < depth; k0 += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
            sa[i / kDepth][i % kDepth] = load_a(i / kDepth, k0 + i % kDepth);
            sb[i / kDepth][i % kDepth] = load_b(i / kDepth, k0 + i % kDepth);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                typename Vec8<T>::type va, vb;
                __builtin_memcpy(&va, &sa[wave / 2 * 32 + i * 16 + lane % 16][lane / 16 * 8], 16);
                __builtin_memcpy(&vb, &sb[wave % 2 * 32 + j * 16 + lane % 16][lane / 16 * 8], 16);
                acc[i][j] = mma(va, vb, acc[i][j]);
            }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                store(wave / 2 * 32 + i * 16 + lane / 16 * 4 + k, wave % 2 * 32 + j * 16 + lane % 16, acc[i][j][k]);
}

template <typename T, bool TRANSPOSED>
__global__ __launch_bounds__(kThreads) void grouped_kernel(Grouped a)
{
    const int64_t out = TRANSPOSED ? a.cols : a.rows, depth = TRANSPOSED ? a.rows : a.cols;
    const int64_t ntiles = (out + kTile - 1) / kTile;
    int64_t mt = blockIdx.x / ntiles;
    const int64_t n0 = blockIdx.x % ntiles * kTile;
    int e = 0;
    int64_t first = 0, end = 0;
    for (;; ++e) {
        if (e == a.experts) return;
        group_range(a, e, first, end);
        const int64_t tiles = (end - first + kTile - 1) / kTile;
        if (mt < tiles) break;
        mt -= tiles;
    }
    const int64_t m0 = first + mt * kTile;
    const T* x = static_cast<const T*>(a.x);
    const T* w = static_cast<const T*>(a.w) + (int64_t)e * a.rows * a.cols;
    T* y = static_cast<T*>(a.y);
    tile_product<T>(
        depth,
        [&](int i, int64_t k) {
            const int64_t r = m0 + i < end ? batch_row(a, m0 + i) : -1;
            return r >= 0 && k < depth ? x[r * a.x_stride + k] : (T)0.0f;
        },
        [&](int j, int64_t k) {
            if (n0 + j >= out || k >= depth) return (T)0.0f;
            return TRANSPOSED ? w[k * a.cols + n0 + j] : w[(n0 + j) * a.cols + k];
        },
        [&](int i, int j, float v) {
            if (m0 + i < end && n0 + j < out) y[(m0 + i) * a.y_stride + n0 + j] = (T)v;
        });
}

template <typename T, typename G>
__global__ __launch_bounds__(kThreads) void grouped_grad_kernel(Grouped a)
{
    const int64_t tr = (a.rows + kTile - 1) / kTile, tc = (a.cols + kTile - 1) / kTile;
    const int e = (int)(blockIdx.x / (tr * tc));
    const int64_t i0 = blockIdx.x / tc % tr * kTile, j0 = blockIdx.x % tc * kTile;
    int64_t first, end;
    group_range(a, e, first, end);
    const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(a.y);
    G* dw = static_cast<G*>(a.dw) + (int64_t)e * a.rows * a.cols;
    tile_product<T>(
        end - first,
        [&](int i, int64_t k) { return i0 + i < a.rows && first + k < end ? dy[(first + k) * a.y_stride + i0 + i] : (T)0.0f; },
        [&](int j, int64_t k) {
            const int64_t r = j0 + j < a.cols && first + k < end ? batch_row(a, first + k) : -1;
            return r >= 0 ? x[r * a.x_stride + j0 + j] : (T)0.0f;
        },
        [&](int i, int j, float v) {
            if (i0 + i >= a.rows || j0 + j >= a.cols) return;
            G* p = dw + (i0 + i) * a.cols + j0 + j;
            *p = (G)(a.accumulate ? v + (float)*p : v);
        });
}

int64_t grouped_blocks(const Grouped& a)
{
    const int64_t out = a.transposed ? a.cols : a.rows;
    return ((a.m + kTile - 1) / kTile + a.experts) * ((out + kTile - 1) / kTile);
}

int64_t grouped_grad_blocks(const Grouped& a)
{
    return (int64_t)a.experts * ((a.rows + kTile - 1) / kTile) * ((a.cols + kTile - 1) / kTile);
}

template <typename T> static void launch_typed(const Grouped& a, hipStream_t stream)
{
    const dim3 grid((unsigned)grouped_blocks(a)), block(kThreads);
    if (a.transposed)
        grouped_kernel<T, true><<<grid, block, 0, stream>>>(a);
    else
        grouped_kernel<T, false><<<grid, block, 0, stream>>>(a);
}

hipError_t launch_grouped_matmul(ElemKind kind, const Grouped& a, hipStream_t stream)
{
    if (kind == kBF16)
        launch_typed<bf16>(a, stream);
    else
        launch_typed<fp16>(a, stream);
    return hipGetLastError();
}

hipError_t launch_grouped_matmul_grad(ElemKind kind, ElemKind grad_kind, const Grouped& a, hipStream_t stream)
{
    const dim3 grid((unsigned)grouped_grad_blocks(a)), block(kThreads);
    if (kind == kBF16) {
        if (grad_kind == kF32)
            grouped_grad_kernel<bf16, float><<<grid, block, 0, stream>>>(a);
        else
            grouped_grad_kernel<bf16, bf16><<<grid, block, 0, stream>>>(a);
    } else {
        if (grad_kind == kF32)
            grouped_grad_kernel<fp16, float><<<grid, block, 0, stream>>>(a);
        else
            grouped_grad_kernel<fp16, fp16><<<grid, block, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace ds
