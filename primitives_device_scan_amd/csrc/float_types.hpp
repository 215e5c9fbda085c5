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

// The 16 bytes of a row from element `at` on, 0 past its end: loaded where they
// are whole and moved down, so that a row's end costs one access, not one per
// element (which made rows of odd length several times slower).
template <typename T>
__device__ __forceinline__ u32x4 load_end(const T* __restrict__ row, int64_t at, int64_t length)
{
    constexpr int N = Vec16<T>::kN;
    if (length < N) {  // uniform
        T t[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            t[i] = row[at + i < length ? at + i : 0];
            if (at + i >= length) __builtin_memset(&t[i], 0, sizeof(T));
        }
        u32x4 v;
        __builtin_memcpy(&v, t, sizeof(v));
        return v;
    }
    const int64_t from = at < length - N ? at : length - N;
    const u32x4 v = *reinterpret_cast<const typename Vec16<T>::type*>(row + from);
    const int64_t over = at - from;
    const int shift = (over < N ? (int)over : N) * (int)sizeof(T) * 8;  // bits
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    if (shift & 64) {
        lo = hi;
        hi = 0;
    }
    const int rest = shift & 63;
    if (rest) {
        lo = lo >> rest | hi << (64 - rest);
        hi >>= rest;
    }
    if (shift >= 128) lo = hi = 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Rounds N floats to T (nearest even) and writes the first `valid` of them.
template <typename T, int N>
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
            *reinterpret_cast<typename Vec16<T>::type*>(p + v * kPer) = u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < valid) p[i] = t[i];
    }
}

}  // namespace ds
