// Element types, activations and the epilogue shared by the layer kernels.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "layers.h"

namespace sgemm {

// ------------------------------------------------------------------ types

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

template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

// One 16-byte access of W elements (or, W = 1, one element), kept as the words
// that were loaded: 16-bit values held one to a register cost registers and
// moves (the norm's backward pass ran at 2.5 TB/s with them).
template <class T, int W>
struct Raw {
    static_assert(W * sizeof(T) == 16, "16-byte accesses");
    uint4 u;
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[W]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (W == 4) {
                f[i] = __uint_as_float(w[i]);
            } else {
                const float2 v = unpack2<T>(w[i]);
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
};
template <class T>
struct Raw<T, 1> {
    T u;
    __device__ __forceinline__ void load(const T *p) { u = *p; }
    __device__ __forceinline__ void zero() { u = from_f32<T>(0.f); }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(u); }
};

// W floats rounded to T and stored as one access.
template <class T, int W>
__device__ __forceinline__ void put(T *p, const float (&f)[W]) {
    if constexpr (W == 1) {
        *p = from_f32<T>(f[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]),
                                                   pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
    }
}

// Asks for the 128-byte line of p in L2.
__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" :: "l"(p));
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

// ------------------------------------------------------------------ launches

// Launches of one call that do not read one another's results (the pieces of a
// plan, the gradients' two products, ...) form a chain, in which a later one fills the
// SMs that the ones before it leave.  The first (kChainNext alone) waits for
// earlier work as ever, and lets the next one start only after that wait: where
// the next one runs, all earlier work has completed.  The others (kChainPrev) do
// not wait at their start but before they end, so that each launch completes after
// the ones before it and the work behind the last one waits for all of them.
// That earlier work has completed says where its results are (L2, at the latest
// when it ended), not that this launch's loads look there: only a launch's own wait
// promises that, and an L1 may hold the same addresses as an earlier call left them
// (workspaces are used again).  So a launch with kChainPrev takes what earlier work
// wrote from L2: by TMA, by __ldcg, or by plain loads after chain_fence, which leaves
// nothing older in the SM's L1; never through the read-only path (__ldg).
__device__ __forceinline__ void chain_begin(int chain) {
    if (!(chain & kChainNext)) pdl_trigger();
    if (!(chain & kChainPrev)) pdl_wait();
    if (chain & kChainNext) pdl_trigger();
}
// (about a microsecond where a launch starts with it, as the planes' does: gradients
// of 500 x 777 x 1001 f32 23.6 us, without it 22.5)
__device__ __forceinline__ void chain_fence(int chain) {
    if (chain & kChainPrev) asm volatile("fence.acq_rel.gpu;" ::: "memory");
}
__device__ __forceinline__ void chain_end(int chain) {
    if (chain & kChainPrev) pdl_wait();
}

// ------------------------------------------------------------------ activations

constexpr float kLog2E = 1.4426950408889634f;

// 1 / (1 + 2^(a b)) by the hardware's power of two and reciprocal (each within a
// few units of 2^-23), formed as 2^-18 / (2^-18 + 2^(a b - 18)): the reciprocal, whose
// results below 2^-126 become 0, is then normal down to a quotient of 2^-144, from
// where on z times it, and the slopes' largest factor (260, tanh form) times it, are
// 0 in bf16 too.  (Without the factor SiLU was 0 from z = -88 on, where bf16 has
// values down to z = -98.)
constexpr float kTailBits = 18.f, kTail = 0x1p-18f;
__device__ __forceinline__ float sigmoid_of_power(float a, float b) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(a, b, -kTailBits)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(kTail + e));
    return r * kTail;
}

// 1 / (1 + exp(-t)).  T is the type that the result is rounded to: for the 16-bit
// types the hardware's approximations (and |t| units of 2^-23 in the exponent) are
// far below its roundoff and take a third of the instructions.  (f32: exp(-|t|), as
// exp(-t) overflows at t = -88.7, where the result is still 3e-39.)
template <class T>
__device__ __forceinline__ float sigmoid(float t) {
    if constexpr (sizeof(T) == 4) {
        const float e = expf(-fabsf(t));
        return (t < 0.f ? e : 1.f) / (1.f + e);
    }
    return sigmoid_of_power(t, -kLog2E);
}

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;   // 1 / sqrt(2 pi)

// The normal distribution's Phi(z) = erfc(-z / sqrt 2) / 2 (1 + erf would lose 4 % of
// it to rounding at z = -5 and all of it from -5.7 on), and the `density`
// exp(-z^2/2), 2^18 times it for the 16-bit types.  For those, with u = |z| and t = 1 / (1 + 0.36 u),
//   Phi(-u) = exp(-u^2/2) t P(t)
// where P, of degree 6, is a least-maximum fit to the smooth rest (over 0 <= u <= 15
// relative error 1.1e-6, 1.3e-6 as evaluated), Phi(u) = 1 - Phi(-u).  (Column sums
// of 4096 x 8192 bf16: 35 us, 78 with erfcf and expf.)  The factor 2^18 keeps
// exp(-z^2/2) normal as far as z Phi(z) is a bf16 number.
template <class T>
__device__ __forceinline__ float normal_cdf(float z, float &density) {
    if constexpr (sizeof(T) == 4) {
        density = expf(-0.5f * z * z);
        return 0.5f * erfcf(-z * kSqrtHalf);
    }
    const float u = fabsf(z);
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.36f, u, 1.f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(density)
        : "f"(fmaf(u * (-0.5f * kLog2E), u, kTailBits)));
    float p = 0.0465225801f * kTail;
    p = fmaf(p, t, -0.177935556f * kTail);
    p = fmaf(p, t, 0.178465992f * kTail);
    p = fmaf(p, t, 0.0282577164f * kTail);
    p = fmaf(p, t, 0.139098883f * kTail);
    p = fmaf(p, t, 0.141884699f * kTail);
    p = fmaf(p, t, 0.143705189f * kTail);
    const float h = density * (t * p);
    return z < 0.f ? h : 1.f - h;
}

// (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), so the tanh form of GELU is z times
// a sigmoid: one exponential and no cancellation near tanh u = -1.
template <class T>
__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case SGEMM_ACT_RELU: return z < 0.f ? 0.f : z;   // a NaN stays one
        case SGEMM_ACT_GELU:
            if constexpr (sizeof(T) == 4)
                return z * sigmoid<T>(2.f * kGeluC * (z + kGeluK * z * z * z));
            else   // the same with the constants multiplied out
                return z * sigmoid_of_power(z, fmaf(z * z, -2.f * kGeluC * kGeluK * kLog2E,
                                                    -2.f * kGeluC * kLog2E));
        case SGEMM_ACT_GELU_ERF: {
            float e;
            return z * normal_cdf<T>(z, e);
        }
        case SGEMM_ACT_SILU: return z * sigmoid<T>(z);
        default: return z;
    }
}

// act of N values; the choice is made once, outside the loop over them.
template <class T, int N>
__device__ __forceinline__ void activate_all(float (&z)[N], int act) {
    if (act == SGEMM_ACT_NONE) return;
    switch (act) {
        case SGEMM_ACT_RELU:
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = activate<T>(z[j], SGEMM_ACT_RELU);
            break;
        case SGEMM_ACT_GELU:
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = activate<T>(z[j], SGEMM_ACT_GELU);
            break;
        case SGEMM_ACT_GELU_ERF:
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = activate<T>(z[j], SGEMM_ACT_GELU_ERF);
            break;
        default:
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = activate<T>(z[j], SGEMM_ACT_SILU);
            break;
    }
}

// z held to -limit .. limit; a NaN stays one.
__device__ __forceinline__ float hold(float z, float limit) {
    float r;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(limit));
    return r;
}

// d act / dz.  With p = (1 + tanh u) / 2: (1 - tanh^2 u) / 2 = 2 p (1 - p).  z is held
// to where the slope has become exactly 0 or 1 in fp32 (p(1 - p) and the density are
// 0 there): beyond, a term that grows with z would meet that 0 as an infinity and
// give NaN (tanh form in 16 bits from |z| = 1.2e13 on, an infinite stored z in all).
template <class T>
__device__ __forceinline__ float activate_grad(float z, int act) {
    switch (act) {
        case SGEMM_ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case SGEMM_ACT_GELU: {
            z = hold(z, 16.f);   // the sigmoid's argument there: 318
            const float z2 = z * z;
            if constexpr (sizeof(T) == 4) {
                const float p = sigmoid<T>(2.f * kGeluC * (z + kGeluK * z2 * z));
                return p + 2.f * kGeluC * z * p * (1.f - p) * (1.f + 3.f * kGeluK * z2);
            } else {   // the same with the constants multiplied out
                const float p = sigmoid_of_power(z, fmaf(z2, -2.f * kGeluC * kGeluK * kLog2E,
                                                         -2.f * kGeluC * kLog2E));
                const float q = z * fmaf(z2, 6.f * kGeluC * kGeluK, 2.f * kGeluC);
                return fmaf(q, fmaf(-p, p, p), p);
            }
        }
        case SGEMM_ACT_GELU_ERF: {
            z = hold(z, 32.f);   // the density's exponent there: -512
            float e;
            const float p = normal_cdf<T>(z, e);
            return fmaf(z * (kRsqrt2Pi * (sizeof(T) == 4 ? 1.f : kTail)), e, p);
        }
        case SGEMM_ACT_SILU: {
            z = hold(z, 256.f);
            const float p = sigmoid<T>(z);
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
    float y = activate<T>(z, e.act);
    if (e.R != nullptr) y += to_f32(static_cast<const T *>(e.R)[row * e.ldr + col]);
    static_cast<T *>(e.Y)[row * e.ldy + col] = from_f32<T>(y);
}

// What the epilogue takes for G fixed columns, loaded once for many rows.
template <class T, int G>
struct ColumnTerms {
    float bias[G], sw[G];
    __device__ __forceinline__ void load(const LayerEpi &e, int col) {
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const bool in = col + j < e.N;
            bias[j] = in && e.bias != nullptr ? to_f32(static_cast<const T *>(e.bias)[col + j]) : 0.f;
            sw[j] = in && e.sw != nullptr ? e.sw[col + j] : 1.f;
        }
    }
};

// Columns col .. col + G - 1 of `row` < M, those below N; one access per matrix
// where the group is whole and e.vec allows it.
template <class T, int G>
__device__ __forceinline__ void finish_group(const LayerEpi &e, const ColumnTerms<T, G> &t, int row,
                                             int col, float (&z)[G]) {
    const bool vec = e.vec >= G && col + G <= e.N;
    T *y = static_cast<T *>(e.Y) + row * e.ldy + col;
    float r[G];
    if (e.R != nullptr) {
        const T *p = static_cast<const T *>(e.R) + row * e.ldr + col;
        if (vec) {
            const Vec<T, G> v = load_vec<T, G>(p);
#pragma unroll
            for (int j = 0; j < G; ++j) r[j] = to_f32(v.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < G; ++j) r[j] = col + j < e.N ? to_f32(p[j]) : 0.f;
        }
    }
    const float sx = e.sx != nullptr ? e.sx[row] : 1.f;
#pragma unroll
    for (int j = 0; j < G; ++j) z[j] = fmaf(z[j], sx * t.sw[j], t.bias[j]);
    auto store = [&](T *p) {
        if (vec) {
            store_vec<T, G>(p, z);
        } else {
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (col + j < e.N) p[j] = from_f32<T>(z[j]);
        }
    };
    if (e.Z != nullptr) store(static_cast<T *>(e.Z) + row * e.ldz + col);
    activate_all<T>(z, e.act);
    if (e.R != nullptr) {
#pragma unroll
        for (int j = 0; j < G; ++j) z[j] += r[j];
    }
    store(y);
}

// One column of R rows from row0 on, the first `rows` of them; the rows'
// residuals are in flight together.
template <class T, int R>
__device__ __forceinline__ void finish_column(const LayerEpi &e, const ColumnTerms<T, 1> &t,
                                              int row0, int rows, int col, float (&z)[R]) {
    float r[R];
    if (e.R != nullptr) {
        const T *p = static_cast<const T *>(e.R) + row0 * e.ldr + col;
#pragma unroll
        for (int i = 0; i < R; ++i) r[i] = i < rows ? to_f32(p[i * e.ldr]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float sx = e.sx != nullptr && i < rows ? e.sx[row0 + i] : 1.f;
        z[i] = fmaf(z[i], sx * t.sw[0], t.bias[0]);
    }
    if (e.Z != nullptr) {
        T *p = static_cast<T *>(e.Z) + row0 * e.ldz + col;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i < rows) p[i * e.ldz] = from_f32<T>(z[i]);
    }
    activate_all<T>(z, e.act);
    T *p = static_cast<T *>(e.Y) + row0 * e.ldy + col;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < rows) p[i * e.ldy] = from_f32<T>(e.R != nullptr ? z[i] + r[i] : z[i]);
}

// 16 values of a 16-bit type as one 32-byte access (aligned to it): a whole
// sector each lane.
__device__ __forceinline__ void load_32b(const void *p, uint32_t (&r)[8]) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p) : "memory");
}

// ------------------------------------------------------------------ f32 planes

// Two values as the three planes' pairs.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&w)[3]) {
    const float x0 = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
    const float y0 = __uint_as_float(__float_as_uint(y) & 0xffff0000u);
    const float rx = x - x0, ry = y - y0;   // exact
    w[0] = (__float_as_uint(x) >> 16) | (__float_as_uint(y) & 0xffff0000u);
    w[1] = pack2<__nv_bfloat16>(rx, ry);
    const float2 m = unpack2<__nv_bfloat16>(w[1]);
    w[2] = pack2<__nv_bfloat16>(rx - m.x, ry - m.y);
}

// W values into the three planes, `plane` elements apart, at `p`.
template <int W>
__device__ __forceinline__ void put_planes(__nv_bfloat16 *p, int64_t plane, const float (&x)[W]) {
    static_assert(W == 1 || W == 4, "one value or four");
    uint32_t w[(W + 1) / 2][3];
#pragma unroll
    for (int i = 0; i < (W + 1) / 2; ++i)
        split_pair(x[2 * i], W == 1 ? 0.f : x[(2 * i + 1) % W], w[i]);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        if constexpr (W == 1)
            *reinterpret_cast<uint16_t *>(p + j * plane) = (uint16_t)w[0][j];
        else
            *reinterpret_cast<uint2 *>(p + j * plane) = make_uint2(w[0][j], w[1][j]);
    }
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
