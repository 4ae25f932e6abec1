// Element types of the operators between the projections: conversion of 16-byte
// (or smaller) groups of fp16, bf16, e4m3 or fp32 elements to and from fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace w4a16 {
namespace elem {

struct E4M3 {
    uint8_t bits;
};

template <typename T>
__device__ __forceinline__ float2 pair_to_f32(uint32_t x);
template <>
__device__ __forceinline__ float2 pair_to_f32<__half>(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}
template <>
__device__ __forceinline__ float2 pair_to_f32<__nv_bfloat16>(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

template <typename T>
__device__ __forceinline__ uint32_t pair_from_f32(float a, float b);
template <>
__device__ __forceinline__ uint32_t pair_from_f32<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pair_from_f32<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Two e4m3 values, the first in the low byte; beyond 448 they saturate, NaN stays.
__device__ __forceinline__ uint16_t pair_to_e4m3(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// The lower and the upper two of four e4m3 values as fp16 (exact).
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

// N consecutive elements to fp32 and back (the address is aligned to their size in
// bytes). Stores of 8 are marked as streaming: what these operators write is read by
// another kernel once. Together with streaming loads that takes residual_rmsnorm from
// 81.8 to 80.1 us (8192 rows of 5120) and rope_append from 23.6 to 22.6 (4099 rows);
// either alone gains nothing.
template <typename T, int N>
struct Vec;

template <int N>
struct Vec16 {  // 16-bit types
    template <typename T>
    static __device__ __forceinline__ void load(const T *p, float (&f)[N]) {
        uint32_t w[N / 2];
        if constexpr (N == 8) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 v = pair_to_f32<T>(w[i]);
            f[2 * i] = v.x, f[2 * i + 1] = v.y;
        }
    }
    template <typename T>
    static __device__ __forceinline__ void store(T *p, const float (&f)[N]) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = pair_from_f32<T>(f[2 * i], f[2 * i + 1]);
        if constexpr (N == 8)
            __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
        else
            *reinterpret_cast<uint32_t *>(p) = w[0];
    }
};
template <int N>
struct Vec<__half, N> : Vec16<N> {};
template <int N>
struct Vec<__nv_bfloat16, N> : Vec16<N> {};
template <>
struct Vec<float, 8> {
    static __device__ __forceinline__ void load(const float *p, float (&f)[8]) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&f)[8]) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
        __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
    }
};
template <int N>
struct Vec<E4M3, N> {
    static __device__ __forceinline__ void store(E4M3 *p, const float (&f)[N]) {
        uint16_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = pair_to_e4m3(f[2 * i], f[2 * i + 1]);
        if constexpr (N == 8)
            __stcs(reinterpret_cast<uint2 *>(p), make_uint2(w[0] | ((uint32_t)w[1] << 16), w[2] | ((uint32_t)w[3] << 16)));
        else
            *reinterpret_cast<uint16_t *>(p) = w[0];
    }
};

}  // namespace elem
}  // namespace w4a16
