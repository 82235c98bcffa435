// Element types, activations and the epilogue shared by the layer kernels.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "layers.h"

namespace sgemm {

// ------------------------------------------------------------------ types

template <class T>
struct TypeOf;
template <>
struct TypeOf<float> {
    static constexpr int id = SGEMM_F32;
};
template <>
struct TypeOf<__nv_bfloat16> {
    static constexpr int id = SGEMM_BF16;
};
template <>
struct TypeOf<__half> {
    static constexpr int id = SGEMM_F16;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
    return __float2half_rn(x);
}

// N consecutive elements as one access of N * sizeof(T) bytes (4, 8 or 16),
// aligned to its size.
template <class T, int N>
struct alignas(N * sizeof(T)) Vec {
    T v[N];
};

template <class T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T *p) {
    return *reinterpret_cast<const Vec<T, N> *>(p);
}

template <class T, int N>
__device__ __forceinline__ void store_vec(T *p, const float (&x)[N]) {
    Vec<T, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = from_f32<T>(x[i]);
    *reinterpret_cast<Vec<T, N> *>(p) = r;
}

// ------------------------------------------------------------------ activations

// 1 / (1 + exp(-t)).  exp(-t) overflows to infinity for t below about -88,
// which gives the limit 0.
__device__ __forceinline__ float sigmoid(float t) { return 1.f / (1.f + expf(-t)); }

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;   // 1 / sqrt(2 pi)

// (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), so the tanh form of GELU is z times
// a sigmoid: one exponential and no cancellation near tanh u = -1.
__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case SGEMM_ACT_RELU: return z < 0.f ? 0.f : z;   // a NaN stays one
        case SGEMM_ACT_GELU: return z * sigmoid(2.f * kGeluC * (z + kGeluK * z * z * z));
        case SGEMM_ACT_GELU_ERF: return 0.5f * z * (1.f + erff(z * kSqrtHalf));
        case SGEMM_ACT_SILU: return z * sigmoid(z);
        default: return z;
    }
}

// d act / dz.  With p = (1 + tanh u) / 2: (1 - tanh^2 u) / 2 = 2 p (1 - p).
__device__ __forceinline__ float activate_grad(float z, int act) {
    switch (act) {
        case SGEMM_ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case SGEMM_ACT_GELU: {
            const float z2 = z * z;
            const float p = sigmoid(2.f * kGeluC * (z + kGeluK * z2 * z));
            return p + 2.f * kGeluC * z * p * (1.f - p) * (1.f + 3.f * kGeluK * z2);
        }
        case SGEMM_ACT_GELU_ERF:
            return 0.5f * (1.f + erff(z * kSqrtHalf)) + z * kRsqrt2Pi * expf(-0.5f * z * z);
        case SGEMM_ACT_SILU: {
            const float p = sigmoid(z);
            return p * (1.f + z * (1.f - p));
        }
        default: return 1.f;
    }
}

// ------------------------------------------------------------------ epilogue

// One element.
template <class T>
__device__ __forceinline__ void finish1(const LayerEpi &e, int row, int col, float acc) {
    float z = acc;
    if (e.sx != nullptr) z *= e.sx[row] * e.sw[col];
    if (e.bias != nullptr) z += to_f32(static_cast<const T *>(e.bias)[col]);
    if (e.Z != nullptr) static_cast<T *>(e.Z)[row * e.ldz + col] = from_f32<T>(z);
    float y = activate(z, e.act);
    if (e.R != nullptr) y += to_f32(static_cast<const T *>(e.R)[row * e.ldr + col]);
    static_cast<T *>(e.Y)[row * e.ldy + col] = from_f32<T>(y);
}

// Columns col .. col + G - 1 (col a multiple of G, G = 4 or 8) of `row` < M,
// those below N; one access per matrix where the group is whole and e.vec
// allows it.
template <class T, int G>
__device__ __forceinline__ void finish(const LayerEpi &e, int row, int col, const float (&acc)[G]) {
    if (e.vec < G || col + G > e.N) {
#pragma unroll
        for (int j = 0; j < G; ++j)
            if (col + j < e.N) finish1<T>(e, row, col + j, acc[j]);
        return;
    }
    float z[G];
#pragma unroll
    for (int j = 0; j < G; ++j) z[j] = acc[j];
    if (e.sx != nullptr) {
        const float sx = e.sx[row];
#pragma unroll
        for (int j = 0; j < G; ++j) z[j] *= sx * e.sw[col + j];
    }
    if (e.bias != nullptr) {
        const Vec<T, G> b = load_vec<T, G>(static_cast<const T *>(e.bias) + col);
#pragma unroll
        for (int j = 0; j < G; ++j) z[j] += to_f32(b.v[j]);
    }
    if (e.Z != nullptr) store_vec<T, G>(static_cast<T *>(e.Z) + row * e.ldz + col, z);
    float y[G];
#pragma unroll
    for (int j = 0; j < G; ++j) y[j] = activate(z[j], e.act);
    if (e.R != nullptr) {
        const Vec<T, G> r = load_vec<T, G>(static_cast<const T *>(e.R) + row * e.ldr + col);
#pragma unroll
        for (int j = 0; j < G; ++j) y[j] += to_f32(r.v[j]);
    }
    store_vec<T, G>(static_cast<T *>(e.Y) + row * e.ldy + col, y);
}

// ------------------------------------------------------------------ 8-bit rows

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 1e-30f;   // keeps 448 / a finite; a row of zeros gets codes 0

// Four values as codes in the bytes of a word: nearest even, saturating at
// +-448, NaN kept.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint8_t to_e4m3(float a) {
    return (uint8_t)__nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float2 from_e4m3x2(uint16_t c) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3);
    return __half22float2(__half2(h));
}

// Larger of two, NaN if either is one (fmaxf drops a NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

}  // namespace sgemm
