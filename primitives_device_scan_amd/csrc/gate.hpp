// gate.hpp -- the gates of the gated recurrence in 32 bits.
//
// A gate a near 1 keeps its state for 1 / (1 - a) steps, and a rounded to 32
// bits is up to 2^-25 off: over 30,000 steps that is 1e-3 of the state, far
// more than the roundings of the state itself (which go both ways). So gates
// that come as sigmoids or exponentials are held as the smaller of a and 1 - a:
// v = a, or v = -(1 - a) where 0.5 <= a <= 1, marked by the sign bit (a = 1 is
// -0.0, a = 0 is +0.0). a h is then v h, plus h where the sign bit is set.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "float_types.hpp"

namespace ds {

enum GateForm { kDecay = 0, kLog = 1, kSigmoid = 2 };

__device__ __forceinline__ bool gate_keeps(float v) { return (int)__builtin_bit_cast(uint32_t, v) < 0; }

// exp(-|g|) to some 2^-23 of itself: the product with log2(e) is taken in two
// parts, since its rounding alone would be |g| 2^-24 of the result, the same
// for every step of a channel whose gate stays where it is. In bf16 (8 bits)
// the product with log2(e) cut to 16 bits is exact.
template <typename T>
__device__ __forceinline__ float exp_minus(float g)
{
    constexpr float kLn2 = 0.69314718f;
    const float m = -__builtin_fabsf(g);
    float e, rest;
    if constexpr (__is_same(T, bf16)) {
        constexpr float kHi = 1.44268798828125f;
        e = __builtin_amdgcn_exp2f(m * kHi);
        rest = m * (float)((1.4426950408889634 - 1.44268798828125) * kLn2);
    } else {
        constexpr float kHi = 1.4426950408889634f;
        const float p = m * kHi;
        e = __builtin_amdgcn_exp2f(p);
        rest = __builtin_fmaf(m, (float)(1.4426950408889634 - (double)kHi), __builtin_fmaf(m, kHi, -p)) * kLn2;
    }
    // far gates' rest may be infinite or NaN where e is 0; a NaN gate is one in e
    return __builtin_fmaf(e, __builtin_amdgcn_fmed3f(rest, -0.002f, 0.002f), e);
}

// v of a gate g that came in type T
template <typename T, GateForm FORM>
__device__ __forceinline__ float gate_of(float g)
{
    if constexpr (FORM == kDecay) return g;
    if constexpr (FORM == kSigmoid) {
        // s = sigmoid(-|g|) <= 0.5: a itself for g < 0, 1 - a otherwise
        const float e = exp_minus<T>(g);
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
        // Below -ln 2 the gate itself, from one rounded product: |g| 2^-24 of it off, but it
        // is below a half, so that no state lives through steps enough to gather that.
        const float near = -__builtin_fabsf(p * g);
        return g <= 0.0f && g > -0.6931f ? near : __builtin_amdgcn_exp2f(g * 1.44269504f);
    }
}

// a h
template <GateForm FORM>
__device__ __forceinline__ float keep_of(float v, float h)
{
    if constexpr (FORM == kDecay) return v * h;
    return __builtin_fmaf(v, h, gate_keeps(v) ? h : 0.0f);
}

// a h + x, or with MIX a h + (1 - a) x, which is h - (1 - a) (h - x) or
// x + a (h - x), whichever has the smaller factor
template <GateForm FORM, bool MIX>
__device__ __forceinline__ float step_of(float v, float h, float x)
{
    if constexpr (FORM == kDecay) return __builtin_fmaf(v, h, MIX ? (1.0f - v) * x : x);
    if constexpr (MIX) return __builtin_fmaf(v, h - x, gate_keeps(v) ? h : x);
    return keep_of<FORM>(v, h) + x;
}

// 1 - a (near 0 for a log gate above 0, a > 1, it has a's own 32 bits)
template <GateForm FORM>
__device__ __forceinline__ float rest_of(float v)
{
    if constexpr (FORM == kDecay) return 1.0f - v;
    return gate_keeps(v) ? -v : 1.0f - v;
}

// The product of gates, in the same form: a near 1 is held as 1 - a, which is the
// sum of (1 - a_t) times the product before; a product of 1,000 gates near 1 that is
// rounded 1,000 times would be 1e-6 off. DECAY (whose gates may be negative) has
// the product alone.
template <GateForm FORM> struct Product {
    float a = 1.0f, rest = 0.0f;
    __device__ __forceinline__ void step(float v)
    {
        // a sigmoid's v > 0 is a gate below 0.5, and so is the product then: `rest` does not count
        if constexpr (FORM == kSigmoid) rest = __builtin_fmaf(-v, a, rest);
        if constexpr (FORM == kLog) rest = __builtin_fmaf(rest_of<FORM>(v), a, rest);
        a = keep_of<FORM>(v, a);
    }
    // v of all of them; NaN stays NaN
    __device__ __forceinline__ float value() const
    {
        if constexpr (FORM == kDecay) return a;
        return a >= 0.5f && a <= 1.0f ? __builtin_copysignf(rest, -1.0f) : __builtin_fabsf(a);
    }
};

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
