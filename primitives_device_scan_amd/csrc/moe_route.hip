// moe_route.hip -- the router of a mixture-of-experts layer: each token's
// top_k experts by logit, their weights, and the gradient of the weights.
//
//   s_e = l_e + bias_e (32 bits); expert e can be chosen where s_e > -inf
//   ids = the top_k experts that can be chosen, by s, ties to the lowest e
//         (-1 past the last one)
//   p_e = softmax of l over the experts that can be chosen, or sigmoid(l_e)
//   w_j = scale * p_ids[j], divided by the sum of the chosen p if `renorm`
//
// One wave per token; lane l holds experts l, l + 64, ... (at most 8).
#include "device_scan.hpp"
#include "float_types.hpp"
#include "launch.hpp"

namespace ds {

constexpr int kRouteMaxPerLane = 8;  // 512 experts

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Largest value of the wave, in every lane. The operands are never NaN. The
// lanes that a step does not reach keep their own value.
__device__ __forceinline__ float wave_max(float x)
{
#define DS_MAX_STEP(CTRL, ROWS)                                                                          \
    x = fmaxf(x, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, x),       \
                                                                       __builtin_bit_cast(int, x), CTRL, \
                                                                       ROWS, 0xf, false)))
    DS_MAX_STEP(0x111, 0xf);
    DS_MAX_STEP(0x112, 0xf);
    DS_MAX_STEP(0x114, 0xf);
    DS_MAX_STEP(0x118, 0xf);
    DS_MAX_STEP(0x142, 0xa);
    DS_MAX_STEP(0x143, 0xc);
#undef DS_MAX_STEP
    return readlane(x, kWave - 1);
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// sigmoid(x) (1 - sigmoid(x)) without the difference from 1, which loses its
// digits for large x; 0 at both infinities.
__device__ __forceinline__ float sigmoid_slope(float x)
{
    const float e = expf(-fabsf(x));
    return e / ((1.0f + e) * (1.0f + e));
}

// Experts per lane is NJ: experts <= 64 * NJ.
template <typename T, int NJ>
__global__ __launch_bounds__(kThreads) void moe_route_kernel(const T* __restrict__ logits, int64_t tokens, int experts,
                                                             int64_t stride, const float* __restrict__ bias,
                                                             int top_k, bool use_sigmoid, bool renorm, float scale,
                                                             float* __restrict__ weights, int32_t* __restrict__ ids)
{
    const int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    if (t >= tokens) return;
    const int lane = lane_id();
    const T* row = logits + t * stride;
    float sel[NJ], top = neg_inf(), total = 0.0f;
    float l[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = j * kWave + lane;
        l[j] = e < experts ? (float)row[e] : neg_inf();
        sel[j] = e < experts && bias ? l[j] + bias[e] : l[j];
        if (!(sel[j] > neg_inf())) sel[j] = l[j] = neg_inf();  // -inf or NaN: never chosen
    }
    if (!use_sigmoid && !renorm) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) top = fmaxf(top, l[j]);
        top = wave_max(top);
#pragma unroll
        for (int j = 0; j < NJ; ++j) total += sel[j] > neg_inf() ? expf(l[j] - top) : 0.0f;
        total = wave_sum(total);
    }
    int mine = -1;              // lane i: the i-th choice
    float chosen = neg_inf();   // and its logit
    for (int i = 0; i < top_k; ++i) {
        float m = sel[0];
#pragma unroll
        for (int j = 1; j < NJ; ++j) m = fmaxf(m, sel[j]);
        m = wave_max(m);
        if (!(m > neg_inf())) break;  // uniform: nothing left
        bool found = false;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint64_t at = ballot(sel[j] == m);
            if (!found && at) {
                found = true;
                const int src = __builtin_ctzll(at);
                const float value = readlane(l[j], src);
                if (lane == i) {
                    mine = j * kWave + src;
                    chosen = value;
                }
                if (lane == src) sel[j] = neg_inf();
            }
        }
    }
    float w = 0.0f;
    if (use_sigmoid) {
        w = mine >= 0 ? sigmoid(chosen) : 0.0f;
    } else {
        if (renorm) top = wave_max(chosen);
        w = mine >= 0 ? expf(chosen - top) : 0.0f;
    }
    if (renorm) total = wave_sum(w);
    if (renorm || !use_sigmoid) w = total > 0.0f || total != total ? w / total : 0.0f;
    if (lane < top_k) {
        weights[t * top_k + lane] = w * scale;
        ids[t * top_k + lane] = mine;
    }
}

// The gradient with respect to the logits, for given ids and d loss / d w:
// the scores are computed again from the logits, then the chain rule goes
// through the division by the chosen scores' sum and through the scores.
template <typename T, int NJ>
__global__ __launch_bounds__(kThreads) void moe_route_grad_kernel(const T* __restrict__ logits, int64_t tokens,
                                                                  int experts, int64_t stride,
                                                                  const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ dweights, int top_k,
                                                                  bool use_sigmoid, bool renorm, float scale,
                                                                  T* __restrict__ dlogits, int64_t dstride)
{
    const int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    if (t >= tokens) return;
    const int lane = lane_id();
    const T* row = logits + t * stride;
    float l[NJ], p[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = j * kWave + lane;
        l[j] = e < experts ? (float)row[e] : neg_inf();
        if (!(l[j] > neg_inf())) l[j] = neg_inf();  // -inf or NaN: no part in the scores
    }
    int id = -1;
    float dw = 0.0f;
    if (lane < top_k) {
        id = ids[t * top_k + lane];
        if (id < 0 || id >= experts) id = -1;
        if (id >= 0) dw = dweights[t * top_k + lane] * scale;
    }
    if (use_sigmoid) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) p[j] = l[j] > neg_inf() ? sigmoid(l[j]) : 0.0f;
    } else {
        float top = l[0], total = 0.0f;
#pragma unroll
        for (int j = 1; j < NJ; ++j) top = fmaxf(top, l[j]);
        top = wave_max(top);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            p[j] = l[j] > neg_inf() ? expf(l[j] - top) : 0.0f;
            total += p[j];
        }
        total = wave_sum(total);
#pragma unroll
        for (int j = 0; j < NJ; ++j) p[j] = total > 0.0f || total != total ? p[j] / total : 0.0f;
    }
    // q: the chosen scores, lane i the i-th
    float q = 0.0f;
    for (int i = 0; i < top_k; ++i) {
        const int e = readlane(id, i);
        if (e < 0) continue;  // uniform
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (e / kWave == j) v = readlane(p[j], e % kWave);
        if (lane == i) q = v;
    }
    if (renorm) {
        float total = wave_sum(q);
        total = total > 0.0f || total != total ? total : 1.0f;
        const float dot = wave_sum(dw * q) / total;
        if (id >= 0) dw = (dw - dot) / total;
    }
    float dp[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) dp[j] = 0.0f;
    for (int i = 0; i < top_k; ++i) {
        const int e = readlane(id, i);
        const float d = readlane(dw, i);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (e == j * kWave + lane) dp[j] += d;
    }
    float dot = 0.0f;
    if (!use_sigmoid) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) dot += dp[j] * p[j];
        dot = wave_sum(dot);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = j * kWave + lane;
        const float d = use_sigmoid ? dp[j] * sigmoid_slope(l[j]) : p[j] * (dp[j] - dot);
        if (e < experts) dlogits[t * dstride + e] = (T)d;
    }
}

int route_max_experts() { return kRouteMaxPerLane * kWave - 1; }
int64_t route_blocks(int64_t tokens) { return (tokens + kWaves - 1) / kWaves; }

template <typename T>
static hipError_t route_typed(const RouteArgs& a, const void* logits, const float* bias, float* weights, int32_t* ids,
                              hipStream_t stream)
{
    const dim3 grid((unsigned)route_blocks(a.tokens)), block(kThreads);
#define DS_ROUTE(NJ)                                                                                         \
    moe_route_kernel<T, NJ><<<grid, block, 0, stream>>>((const T*)logits, a.tokens, a.experts, a.stride, bias, \
                                                        a.top_k, a.use_sigmoid, a.renorm, a.scale, weights, ids)
    if (a.experts <= kWave) DS_ROUTE(1);
    else if (a.experts <= 2 * kWave) DS_ROUTE(2);
    else if (a.experts <= 4 * kWave) DS_ROUTE(4);
    else DS_ROUTE(8);
#undef DS_ROUTE
    return hipGetLastError();
}

template <typename T>
static hipError_t route_grad_typed(const RouteArgs& a, const void* logits, const int32_t* ids, const float* dweights,
                                   void* dlogits, int64_t dstride, hipStream_t stream)
{
    const dim3 grid((unsigned)route_blocks(a.tokens)), block(kThreads);
#define DS_ROUTE(NJ)                                                                                           \
    moe_route_grad_kernel<T, NJ><<<grid, block, 0, stream>>>((const T*)logits, a.tokens, a.experts, a.stride, ids, \
                                                             dweights, a.top_k, a.use_sigmoid, a.renorm, a.scale, \
                                                             (T*)dlogits, dstride)
    if (a.experts <= kWave) DS_ROUTE(1);
    else if (a.experts <= 2 * kWave) DS_ROUTE(2);
    else if (a.experts <= 4 * kWave) DS_ROUTE(4);
    else DS_ROUTE(8);
#undef DS_ROUTE
    return hipGetLastError();
}

hipError_t launch_moe_route(ElemKind kind, const RouteArgs& a, const void* logits, const float* bias, float* weights,
                            int32_t* ids, hipStream_t stream)
{
    switch (kind) {
    case kF32: return route_typed<float>(a, logits, bias, weights, ids, stream);
    case kBF16: return route_typed<bf16>(a, logits, bias, weights, ids, stream);
    case kF16: return route_typed<fp16>(a, logits, bias, weights, ids, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_moe_route_grad(ElemKind kind, const RouteArgs& a, const void* logits, const int32_t* ids,
                                 const float* dweights, void* dlogits, int64_t dstride, hipStream_t stream)
{
    switch (kind) {
    case kF32: return route_grad_typed<float>(a, logits, ids, dweights, dlogits, dstride, stream);
    case kBF16: return route_grad_typed<bf16>(a, logits, ids, dweights, dlogits, dstride, stream);
    case kF16: return route_grad_typed<fp16>(a, logits, ids, dweights, dlogits, dstride, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ds
