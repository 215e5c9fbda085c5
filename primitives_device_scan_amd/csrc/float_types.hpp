// float_types.hpp -- the floating types of the language-model operators: their
// storage, 16-byte vectors at any element alignment, and conversion to and
// from the 32-bit values that all sums are held in.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tile.hpp"

namespace ds {

typedef __bf16 bf16;
typedef _Float16 fp16;
struct fp8 {  // e4m3, no infinities, NaN 0x7f / 0xff
    uint8_t bits;
};

// 16 bytes of T at an address that is aligned to T alone (rows of odd width,
// slices): global accesses of any alignment are one instruction here, so one
// code path serves every pointer; a wave's run then touches one more line.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
template <int BYTES> struct VecAligned;
template <> struct VecAligned<4> { using type = u32x4_a4; };
template <> struct VecAligned<2> { using type = u32x4_a2; };
template <> struct VecAligned<1> { using type = u32x4_a1; };
template <typename T> struct Vec16 {
    static constexpr int kN = kVecBytes / (int)sizeof(T);
    using type = typename VecAligned<(int)sizeof(T)>::type;
};

// N values of T starting at p, as 32-bit floats (exact for every type). Only
// the first `valid` are read where `valid` < N; the others are 0.
template <typename T, int N>
__device__ __forceinline__ void load_floats(const T* __restrict__ p, int64_t valid, float (&x)[N])
{
    static_assert(N == Vec16<T>::kN, "one 16-byte access");
    if (valid >= N) {
        const u32x4 v = *reinterpret_cast<const typename Vec16<T>::type*>(p);
        T t[N];
        __builtin_memcpy(t, &v, sizeof(t));
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = (float)t[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = i < valid ? (float)p[i] : 0.0f;
    }
}

// Rounds N floats to T (nearest even) and writes the first `valid` of them
// (NT: past the cache).
template <typename T, int N, bool NT = false>
__device__ __forceinline__ void store_floats(T* __restrict__ p, int64_t valid, const float (&x)[N])
{
    constexpr int kPer = Vec16<T>::kN;
    static_assert(N % kPer == 0, "whole 16-byte accesses");
    T t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = (T)x[i];
    if (valid >= N) {
#pragma unroll
        for (int v = 0; v < N / kPer; ++v) {
            u32x4 u;
            __builtin_memcpy(&u, t + v * kPer, sizeof(u));
            if constexpr (NT)
                __builtin_nontemporal_store(u, reinterpret_cast<typename Vec16<T>::type*>(p + v * kPer));
            else
                *reinterpret_cast<typename Vec16<T>::type*>(p + v * kPer) = u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < valid) p[i] = t[i];
    }
}

}  // namespace ds
