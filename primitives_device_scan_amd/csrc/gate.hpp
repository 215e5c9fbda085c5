// gate.hpp -- the gates of the gated recurrence in 32 bits.
//
// A gate a near 1 keeps its state for 1 / (1 - a) steps, and a rounded to 32
// bits is up to 2^-25 off: over 30,000 steps that is 1e-3 of the state, far
// more than the roundings of the state itself (which go both ways). So gates
// that come as sigmoids or exponentials are held as the smaller of a and 1 - a:
// v = a, or v = -(1 - a) where 0.5 <= a <= 1, marked by the sign bit (a = 1 is
// -0.0). A step is then fma(v, h, b), plus h where the sign bit is set.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ds {

enum GateForm { kDecay = 0, kLog = 1, kSigmoid = 2 };

__device__ __forceinline__ bool gate_keeps(float v) { return (int)__builtin_bit_cast(uint32_t, v) < 0; }

template <GateForm FORM>
__device__ __forceinline__ float gate_of(float g)
{
    constexpr float kLog2e = 1.44269504f;
    if constexpr (FORM == kDecay) return g;
    if constexpr (FORM == kSigmoid) {
        // s = sigmoid(-|g|) <= 0.5: a itself for g < 0, 1 - a otherwise
        const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(g) * kLog2e);
        return __builtin_copysignf(e * __builtin_amdgcn_rcpf(1.0f + e), -g);
    }
    if constexpr (FORM == kLog) {
        // expm1(g) / g on [-ln 2, 0] by its power series: the first term left
        // out is below 2^-24 of the sum
        float p = 1.0f / 3628800.0f;
        p = __builtin_fmaf(p, g, 1.0f / 362880.0f);
        p = __builtin_fmaf(p, g, 1.0f / 40320.0f);
        p = __builtin_fmaf(p, g, 1.0f / 5040.0f);
        p = __builtin_fmaf(p, g, 1.0f / 720.0f);
        p = __builtin_fmaf(p, g, 1.0f / 120.0f);
        p = __builtin_fmaf(p, g, 1.0f / 24.0f);
        p = __builtin_fmaf(p, g, 1.0f / 6.0f);
        p = __builtin_fmaf(p, g, 0.5f);
        p = __builtin_fmaf(p, g, 1.0f);
        const float near = -__builtin_fabsf(p * g);
        return g <= 0.0f && g > -0.6931f ? near : __builtin_amdgcn_exp2f(g * kLog2e);
    }
}

// a h + b
template <GateForm FORM>
__device__ __forceinline__ float step_of(float v, float h, float b)
{
    const float y = __builtin_fmaf(v, h, b);
    if constexpr (FORM == kDecay) return y;
    return y + (gate_keeps(v) ? h : 0.0f);
}

// 1 - a (near 0 for a log gate above 0, a > 1, it has a's own 32 bits)
template <GateForm FORM>
__device__ __forceinline__ float rest_of(float v)
{
    if constexpr (FORM == kDecay) return 1.0f - v;
    return gate_keeps(v) ? -v : 1.0f - v;
}

// d a / d g
template <GateForm FORM>
__device__ __forceinline__ float slope_of(float v)
{
    if constexpr (FORM == kDecay) return 1.0f;
    const float s = __builtin_fabsf(v);
    if constexpr (FORM == kSigmoid) return s * (1.0f - s);
    return gate_keeps(v) ? 1.0f + v : v;
}

}  // namespace ds
