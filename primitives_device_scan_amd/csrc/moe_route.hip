// moe_route.hip -- the router of a mixture-of-experts layer: each token's
// top_k experts by logit, their weights, and the gradient of the weights.
//
//   s_e = l_e + bias_e (32 bits); expert e can be chosen where s_e > -inf
//   ids = the top_k experts that can be chosen, by s, ties to the lowest e
//         (-1 past the last one)
//   p_e = softmax of l over the experts that can be chosen, or sigmoid(l_e)
//   w_j = scale * p_ids[j], divided by the sum of the chosen p if `renorm`
//
// A token is a group of L lanes, so a wave works on 64 / L tokens at once: with
// a wave to a token the instructions of the selection were what bounded it.
#include "device_scan.hpp"
#include "float_types.hpp"
#include "launch.hpp"

namespace ds {

constexpr int kMostExperts = 511;
constexpr int kMostTopK = 64;
typedef float f32x4_v __attribute__((ext_vector_type(4)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_swap(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, true);  // every lane has a source
}

// x combined over the group's L lanes, in every one of them: neighbours, pairs,
// then mirrored halves of 8 and of 16 lanes.
template <int L, typename OP>
__device__ __forceinline__ uint32_t group_all(uint32_t x, OP op)
{
    x = op(x, dpp_swap<0xB1>(x));
    x = op(x, dpp_swap<0x4E>(x));
    if constexpr (L >= 8) x = op(x, dpp_swap<0x141>(x));
    if constexpr (L >= 16) x = op(x, dpp_swap<0x140>(x));
    return x;
}
template <int L> __device__ __forceinline__ uint32_t group_max(uint32_t x)
{
    return group_all<L>(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L> __device__ __forceinline__ uint32_t group_min(uint32_t x)
{
    return group_all<L>(x, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int L> __device__ __forceinline__ float group_sum(float x)
{
    return __builtin_bit_cast(float, group_all<L>(__builtin_bit_cast(uint32_t, x), [](uint32_t a, uint32_t b) {
                                  return __builtin_bit_cast(
                                      uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
                              }));
}

// Floats as whole numbers of the same order, both zeros alike and NaN as -inf;
// 0 is below every float. (The sum makes -0 a +0 and every NaN a quiet one,
// which the maximum then drops.)
constexpr uint32_t kNoKey = 0x007FFFFFu;  // of -inf
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, fmaxf(x + 0.0f, neg_inf()));
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __builtin_bit_cast(float, k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
template <int L> __device__ __forceinline__ float group_max(float x) { return key_value(group_max<L>(order_key(x))); }

// By the exponential that does not overflow, so that scores go down to 2^-149.
__device__ __forceinline__ float sigmoid(float x)
{
    const float e = expf(-fabsf(x));
    return (x >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// Shares of chosen scores, whose largest logit is `top`. Softmax scores are
// exp(x - top) up to a factor that the division takes away, and so are sigmoid
// scores where all are small (1 + e^x is 1 in 32 bits), which keeps their bits
// where the scores themselves run out of them. Below kNoScore a sigmoid rounds
// to 0 in 32 bits: no share.
constexpr float kSmallScore = -80.0f;
constexpr float kNoScore = -103.9721f;  // ln 2^-150
__device__ __forceinline__ float share_score(float x, float top, bool use_sigmoid)
{
    if (use_sigmoid && top >= kSmallScore) return sigmoid(x);
    return use_sigmoid && top < kNoScore ? 0.0f : expf(x - top);
}

// exp(x) for the router's sum over all experts: 2^(x log2 e), off by at most
// 1.5 |x| + 2 steps of 2^-24, relative (the product's two roundings), where the
// library function takes five times the instructions; 0 below 2^-126. In a sum
// that has a term of 1 that is at most a step per term.
__device__ __forceinline__ float exp_sum(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// exp(x) for the gradient, x <= 0, where it is each element's own factor: what
// the product x log2 e loses, and log2 e as a float, is put back, since 2^(t + r)
// = 2^t (1 + r ln 2) for small r: 3 steps. Where the gradient is rounded to 16
// bits, exp_sum: its 130 steps at most are a thirtieth of that rounding in fp16,
// less in bf16. (65,536 tokens of 256 experts, no renormalising: fp32 25.7 us
// with exp_sum, 26.6 with this; bf16 15.9 and 17.4.)
template <typename T>
__device__ __forceinline__ float exp_factor(float x)
{
    if constexpr (sizeof(T) == 2) return exp_sum(x);
    x = x < -200.0f ? -200.0f : x;  // 0 all the same, and t stays finite
    const float t = x * 1.44269504f, r = __builtin_fmaf(x, 1.925963e-8f, __builtin_fmaf(x, 1.44269504f, -t));
    const float p = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(p, r * 0.693147181f, p);
}

// sigmoid(x) (1 - sigmoid(x)) without the difference from 1, which loses its
// digits for large x; 0 at both infinities.
__device__ __forceinline__ float sigmoid_slope(float x)
{
    const float e = expf(-fabsf(x));
    return e / ((1.0f + e) * (1.0f + e));
}

// This lane's logits of its token: vector v holds experts (v * L + lane) * N ..
// + N - 1, so that a group's loads are whole lines; -inf past the last expert.
template <typename T, int L, int NV>
__device__ __forceinline__ void load_logits(const T* __restrict__ row, int experts, int lane,
                                            float (&l)[NV][Vec16<T>::kN])
{
    constexpr int N = Vec16<T>::kN;
    if (experts % N == 0) {
        u32x4 raw[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int e = (v * L + lane) * N;
            raw[v] = *reinterpret_cast<const typename Vec16<T>::type*>(row + (e < experts ? e : 0));
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            T t[N];
            __builtin_memcpy(t, &raw[v], sizeof(t));
#pragma unroll
            for (int j = 0; j < N; ++j) l[v][j] = (v * L + lane) * N < experts ? (float)t[j] : neg_inf();
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int e = (v * L + lane) * N + j;
                l[v][j] = e < experts ? (float)row[e] : neg_inf();
            }
    }
}

// The bias of experts e0 .. e0 + N - 1 (any value past the last expert).
template <int N>
__device__ __forceinline__ void load_bias(const float* __restrict__ bias, int e0, int experts, float (&b)[N])
{
    if (experts % N == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const f32x4_v v = *reinterpret_cast<const f32x4_a4*>(bias + (e0 < experts ? e0 : 0) + j);
#pragma unroll
            for (int i = 0; i < 4; ++i) b[j + i] = v[i];
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) b[j] = bias[e0 + j < experts ? e0 + j : 0];
    }
}

// ---------------------------------------------------------------------------
// Selection. A token's keys lie in LDS, in strips of S consecutive experts; lane
// i of the group knows the largest key of strip i. A choice finds the largest
// of these, the strip that has it (the first, so ties go to the lowest expert),
// then the group reads that strip, S / L keys to a lane, finds the expert and
// the strip's next largest key. 65,536 tokens, top-8 of 256, bf16 with a bias:
// see the launcher.
// ---------------------------------------------------------------------------
template <typename T, int L, int S>
__global__ __launch_bounds__(kThreads) void moe_route_kernel(const T* __restrict__ logits, int64_t tokens, int experts,
                                                             int64_t stride, const float* __restrict__ bias,
                                                             int top_k, bool use_sigmoid, bool renorm, float scale,
                                                             float* __restrict__ weights, int32_t* __restrict__ ids)
{
    constexpr int N = Vec16<T>::kN, NV = (S + N - 1) / N, P = S / L;
    constexpr int kStrip = S + 4;  // words; the padding puts the strips' equal places into different banks
    constexpr int kGroups = kWave / L;
    static_assert(S % N == 0 && S % L == 0 && S >= 4, "whole vectors to a strip, whole shares to a lane");
    __shared__ __align__(16) uint32_t s_key[kWaves][kGroups][L * kStrip];
    __shared__ uint16_t s_id[kWaves][kGroups][kMostTopK];
    constexpr uint16_t kNone = 0xFFFF;
    static_assert(L * kStrip >= (L * S < kMostTopK ? L * S : kMostTopK), "the keys' place holds the chosen scores");
    const int wave = threadIdx.x / kWave, group = lane_id() / L, lane = lane_id() % L;
    const int64_t t = ((int64_t)blockIdx.x * kWaves + wave) * kGroups + group;
    const bool there = t < tokens;
    const T* row = logits + (there ? t : tokens - 1) * stride;
    uint32_t* keys = s_key[wave][group];
    uint16_t* choice = s_id[wave][group];

    float l[NV][N];
    load_logits<T, L, NV>(row, experts, lane, l);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e0 = (v * L + lane) * N;
        float sel[N];
#pragma unroll
        for (int j = 0; j < N; ++j) sel[j] = l[v][j];
        if (bias) {
            float b[N];
            load_bias<N>(bias, e0, experts, b);
#pragma unroll
            for (int j = 0; j < N; ++j) sel[j] += b[j];
        }
        // -inf past the last expert, but +inf + -inf is NaN: both keys are kNoKey, which is never chosen
        uint32_t* at = keys + e0 / S * kStrip + e0 % S;
#pragma unroll
        for (int j = 0; j < N; j += 4)
            *reinterpret_cast<u32x4*>(at + j) =
                u32x4{order_key(sel[j]), order_key(sel[j + 1]), order_key(sel[j + 2]), order_key(sel[j + 3])};
    }
    float top = 0.0f, total = 0.0f;
    if (!use_sigmoid && !renorm) {  // over the experts that can be chosen
        top = neg_inf();
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int e0 = (v * L + lane) * N;
            const uint32_t* at = keys + e0 / S * kStrip + e0 % S;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (at[j] <= kNoKey) l[v][j] = neg_inf();
                top = l[v][j] > top ? l[v][j] : top;
            }
        }
        top = group_max<L>(top);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j) total += l[v][j] > neg_inf() ? exp_sum(l[v][j] - top) : 0.0f;
        total = group_sum<L>(total);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    uint32_t best = 0;  // largest key of this lane's strip
#pragma unroll
    for (int j = 0; j < S; j += 4) {
        const u32x4 k = *reinterpret_cast<const u32x4*>(keys + lane * kStrip + j);
#pragma unroll
        for (int q = 0; q < 4; ++q) best = k[q] > best ? k[q] : best;
    }
    for (int i = 0; i < top_k; ++i) {
        const uint32_t m = group_max<L>(best);
        const uint32_t w = group_min<L>(best == m ? (uint32_t)lane : (uint32_t)L);
        uint32_t* strip = keys + w * kStrip;
        uint32_t x[P], at = S;
#pragma unroll
        for (int q = 0; q < P; ++q) x[q] = strip[lane * P + q];
#pragma unroll
        for (int q = P - 1; q >= 0; --q) at = x[q] == m ? (uint32_t)(lane * P + q) : at;
        at = group_min<L>(at);
        uint32_t next = 0;
#pragma unroll
        for (int q = 0; q < P; ++q) next = (uint32_t)(lane * P + q) != at && x[q] > next ? x[q] : next;
        next = group_max<L>(next);
        if ((uint32_t)lane == w) best = next;
        if (lane == 0) {
            strip[at] = 0u;
            choice[i] = m > kNoKey ? (uint16_t)(w * S + at) : kNone;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // the chosen logits, their scores, the weights
    float* chosen = reinterpret_cast<float*>(keys);  // no key is needed any more
    float most = neg_inf();
    for (int j = lane; j < top_k; j += L) {
        const uint16_t id = choice[j];
        const float x = id != kNone ? (float)row[id] : neg_inf();
        chosen[j] = x;
        most = x > most ? x : most;
    }
    if (renorm) top = group_max<L>(most);
    float sum = 0.0f;
    for (int j = lane; j < top_k; j += L) {
        const float x = chosen[j];
        const float p = choice[j] == kNone ? 0.0f
                        : renorm           ? share_score(x, top, use_sigmoid)
                        : use_sigmoid      ? sigmoid(x)
                                           : expf(x - top);
        chosen[j] = p;
        sum += p;
    }
    if (renorm) total = group_sum<L>(sum);
    for (int j = lane; j < top_k; j += L) {
        float w = chosen[j];
        if (renorm || !use_sigmoid) w = total > 0.0f || total != total ? w / total : 0.0f;
        if (there) {
            weights[t * top_k + j] = w * scale;
            ids[t * top_k + j] = choice[j] == kNone ? -1 : choice[j];
        }
    }
}

// ---------------------------------------------------------------------------
// The gradient with respect to the logits, for given ids and d loss / d w:
// the scores are computed again from the logits, then the chain rule goes
// through the division by the chosen scores' sum and through the scores. With
// renorm the two give
//   d / d l_e = sum over j with ids[j] = e of w_j (dw_j - sum_i w_i dw_i),
// times 1 - sigmoid(l_e) for sigmoid scores: the other logits are not read
// (they have no part, however much larger they are) and get 0. The chosen
// experts' parts are added up in LDS, choice by choice, so an expert that is
// named twice has its parts added in their order.
// The bias is the router's: it says which experts can be chosen, no more.
// Bound by memory: 65,536 tokens of 256 experts in fp32, top-8: softmax 19.9 us
// with renorm (the rows written and a line per chosen logit), 26.6 us without
// (138 MB at 5.2 TB/s; 51 us with a wave to a token); sigmoid 19.9-20.2.
// ---------------------------------------------------------------------------
template <typename T, int L, int NV>
__global__ __launch_bounds__(kThreads) void moe_route_grad_kernel(const T* __restrict__ logits, int64_t tokens,
                                                                  int experts, int64_t stride,
                                                                  const float* __restrict__ bias,
                                                                  const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ dweights, int top_k,
                                                                  bool use_sigmoid, bool renorm, float scale,
                                                                  T* __restrict__ dlogits, int64_t dstride)
{
    constexpr int N = Vec16<T>::kN, kGroups = kWave / L, M = kMostTopK / L;
    __shared__ __align__(16) float s_dp[kWaves][kGroups][NV * L * N];
    const int wave = threadIdx.x / kWave, group = lane_id() / L, lane = lane_id() % L;
    const int64_t t = ((int64_t)blockIdx.x * kWaves + wave) * kGroups + group;
    const bool there = t < tokens;
    const int64_t token = there ? t : tokens - 1;
    const T* row = logits + token * stride;
    float* dp = s_dp[wave][group];
    // choice j is held by lane j % L, as its (j / L)-th
    int id[M];
    float dw[M], q[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        id[m] = -1;
        dw[m] = q[m] = 0.0f;
        if (m * L < top_k) {  // uniform
            const int j = m * L + lane;
            if (j < top_k) {
                id[m] = ids[token * top_k + j];
                dw[m] = dweights[token * top_k + j] * scale;
            }
            if (id[m] < 0 || id[m] >= experts) id[m] = -1;
        }
    }
    // a choice of what cannot be chosen is none: it has no score, and its dw is not looked at
    float l[NV][N], total = 0.0f;
    float chosen[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        chosen[m] = m * L < top_k && id[m] >= 0 ? (float)row[id[m]] : neg_inf();
        const float s = bias && m * L < top_k && id[m] >= 0 ? chosen[m] + bias[id[m]] : chosen[m];
        if (!(s > neg_inf())) {
            id[m] = -1;
            dw[m] = 0.0f;
            chosen[m] = neg_inf();
        }
    }
    float top = neg_inf();
    if (renorm) {
#pragma unroll
        for (int m = 0; m < M; ++m) top = chosen[m] > top ? chosen[m] : top;  // false for NaN
        top = group_max<L>(top);
    } else if (!use_sigmoid) {
        load_logits<T, L, NV>(row, experts, lane, l);
        if (bias) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int e0 = (v * L + lane) * N;
                float b[N];
                load_bias<N>(bias, e0, experts, b);
#pragma unroll
                for (int j = 0; j < N; ++j) l[v][j] = l[v][j] + b[j] > neg_inf() ? l[v][j] : neg_inf();
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j) top = l[v][j] > top ? l[v][j] : top;  // false for NaN
        top = group_max<L>(top);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                l[v][j] = l[v][j] > neg_inf() ? exp_factor<T>(l[v][j] - top) : 0.0f;
                total += l[v][j];
            }
        total = group_sum<L>(total);
        total = total > 0.0f || total != total ? 1.0f / total : 0.0f;
    }
    // the chosen scores; with renorm as share_score gives them
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m)
        if (m * L < top_k) {
            if (id[m] >= 0)
                q[m] = renorm        ? share_score(chosen[m], top, use_sigmoid)
                       : use_sigmoid ? sigmoid(chosen[m])
                                     : exp_factor<T>(chosen[m] - top) * total;
            sum += q[m];
        }
    if (renorm) {  // shares, and dw less its mean over them; the sum may be too small for dw to be divided by it
        sum = group_sum<L>(sum);
        sum = sum > 0.0f || sum != sum ? sum : 1.0f;
#pragma unroll
        for (int m = 0; m < M; ++m)
            if (m * L < top_k) {
                q[m] /= sum;
                dot += dw[m] * q[m];
            }
        dot = group_sum<L>(dot);
#pragma unroll
        for (int m = 0; m < M; ++m)
            if (id[m] >= 0) dw[m] -= dot;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < N; j += 4) *reinterpret_cast<f32x4_v*>(dp + (v * L + lane) * N + j) = f32x4_v{0.0f, 0.0f, 0.0f, 0.0f};
    float all = 0.0f;  // softmax: the part that every expert has, sum of dp p
#pragma unroll
    for (int m = 0; m < M; ++m)
        if (m * L < top_k) {
            float d = dw[m];
            if (renorm) d *= use_sigmoid ? q[m] / (1.0f + expf(chosen[m])) : q[m];  // 1 - sigmoid: d log sigmoid
            else if (use_sigmoid) d *= sigmoid_slope(chosen[m]);
            all += dw[m] * q[m];
            for (int i = 0; i < L && m * L + i < top_k; ++i)
                if (lane == i && id[m] >= 0)
                    __hip_atomic_fetch_add(dp + id[m], d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
    if (!use_sigmoid && !renorm) all = group_sum<L>(all);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    T* out = dlogits + token * dstride;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e0 = (v * L + lane) * N;
        float d[N];
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const f32x4_v x = *reinterpret_cast<const f32x4_v*>(dp + e0 + j);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[j + i] = x[i];
        }
        if (!use_sigmoid && !renorm) {
#pragma unroll
            for (int j = 0; j < N; ++j) d[j] = l[v][j] * total * (d[j] - all);
        }
        if (there && e0 < experts) store_floats<T, N>(out + e0, experts - e0, d);
    }
}

int route_max_experts() { return kMostExperts; }
int64_t route_blocks(int64_t tokens) { return (tokens + kWaves - 1) / kWaves; }  // of the largest launch, or more

// Lanes to a token: as few as the keys of a wave's tokens leave LDS for (four
// workgroups to a CU at 256 experts). 65,536 tokens, top-8 of 256 in bf16 with
// a bias and sigmoid scores: 17.0-17.8 us, where the bytes take 6.1. What bounds
// it are the selection's instructions, about 65 per choice for a wave's eight
// tokens (20 of them waits between dependent lane moves): vector instructions
// are issued in 0.66 of the time, and the waves wait in 0.56 of theirs. A wave
// to a token took 51.6 us.
template <typename T>
static hipError_t route_typed(const RouteArgs& a, const void* logits, const float* bias, float* weights, int32_t* ids,
                              hipStream_t stream)
{
    const auto launch = [&](auto kernel, int lanes) {
        const int64_t per_block = kWaves * (kWave / lanes);
        kernel<<<dim3((unsigned)((a.tokens + per_block - 1) / per_block)), dim3(kThreads), 0, stream>>>(
            (const T*)logits, a.tokens, a.experts, a.stride, bias, a.top_k, a.use_sigmoid, a.renorm, a.scale, weights,
            ids);
        return hipGetLastError();
    };
    if (a.experts <= 32) return launch(moe_route_kernel<T, 4, 8>, 4);
    if (a.experts <= 64) return launch(moe_route_kernel<T, 4, 16>, 4);
    if (a.experts <= 128) return launch(moe_route_kernel<T, 8, 16>, 8);
    if (a.experts <= 256) return launch(moe_route_kernel<T, 8, 32>, 8);
    return launch(moe_route_kernel<T, 16, 32>, 16);
}

template <typename T>
static hipError_t route_grad_typed(const RouteArgs& a, const void* logits, const float* bias, const int32_t* ids,
                                   const float* dweights, void* dlogits, int64_t dstride, hipStream_t stream)
{
    constexpr int W = 16 / Vec16<T>::kN;  // vectors for 16 experts to a lane
    const auto launch = [&](auto kernel, int lanes) {
        const int64_t per_block = kWaves * (kWave / lanes);
        kernel<<<dim3((unsigned)((a.tokens + per_block - 1) / per_block)), dim3(kThreads), 0, stream>>>(
            (const T*)logits, a.tokens, a.experts, a.stride, bias, ids, dweights, a.top_k, a.use_sigmoid, a.renorm,
            a.scale, (T*)dlogits, dstride);
        return hipGetLastError();
    };
    if (a.experts <= 64) return launch(moe_route_grad_kernel<T, 8, W / 2>, 8);
    if (a.experts <= 128) return launch(moe_route_grad_kernel<T, 8, W>, 8);
    if (a.experts <= 256) return launch(moe_route_grad_kernel<T, 16, W>, 16);
    return launch(moe_route_grad_kernel<T, 16, 2 * W>, 16);
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

hipError_t launch_moe_route_grad(ElemKind kind, const RouteArgs& a, const void* logits, const float* bias,
                                 const int32_t* ids, const float* dweights, void* dlogits, int64_t dstride,
                                 hipStream_t stream)
{
    switch (kind) {
    case kF32: return route_grad_typed<float>(a, logits, bias, ids, dweights, dlogits, dstride, stream);
    case kBF16: return route_grad_typed<bf16>(a, logits, bias, ids, dweights, dlogits, dstride, stream);
    case kF16: return route_grad_typed<fp16>(a, logits, bias, ids, dweights, dlogits, dstride, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ds
