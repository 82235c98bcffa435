// Shared by the row norms (norm.cu, layernorm.cu): loads of a row's pieces, 8-bit stores, the
// shape of the row groups and their launch.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "layer_math.cuh"
#include "layers.h"

namespace sgemm {
namespace norm {

constexpr int kMaxThreads = 1024;

// (sum, max) of every row group of the CTA, the same values in each of its
// threads.  red: 32 float2 of shared memory, not in use since the CTA's last
// barrier but one.
__device__ __forceinline__ float2 group_reduce(float sum, float top, float2 *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    const int warps = blockDim.x >> 5;   // of one group
    if (warps == 1) return make_float2(sum, top);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2 *mine = red + threadIdx.y * warps;
    if (lane == 0) mine[warp] = make_float2(sum, top);
    __syncthreads();
    const float2 p = lane < warps ? mine[lane] : make_float2(0.f, 0.f);
    sum = p.x;
    top = p.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    return make_float2(sum, top);
}

// W elements from p, or zeros.
template <class T, int W>
__device__ __forceinline__ Raw<T, W> load_or_zero(const T *p, bool in) {
    Raw<T, W> v;
    if (in)
        v.load(p);
    else
        v.zero();
    return v;
}

template <int W>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&y)[W]) {
    if constexpr (W == 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(to_e4m3x4(y[0], y[1], y[2], y[3]),
                                                   to_e4m3x4(y[4], y[5], y[6], y[7]));
    } else if constexpr (W == 4) {
        *reinterpret_cast<uint32_t *>(p) = to_e4m3x4(y[0], y[1], y[2], y[3]);
    } else if constexpr (W == 2) {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)to_e4m3x4(y[0], y[1], 0.f, 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) p[i] = to_e4m3(y[i]);
    }
}

// ------------------------------------------------------------------ host side

// Threads of a row group and groups of a CTA for n accesses a row, nv a
// thread; tpr 0 when the row does not fit a group.
struct Shape {
    int tpr, groups;
};
inline Shape shape_for(int64_t n, int nv) {
    const int64_t per = (n + nv - 1) / nv;
    if (per > kMaxThreads) return {0, 0};
    Shape s;
    s.tpr = per <= 32 ? 32 : (int)((per + 31) / 32 * 32);
    s.groups = s.tpr >= 256 ? 1 : 256 / s.tpr;
    return s;
}

// Elements of the widest access (16, 8 or 4 bytes, or one element) that rows of D elements allow:
// what every base and leading dimension (of `size`-byte elements; an 8-bit output's of one byte
// an element) is a multiple of.
inline bool aligned_to(const void *p, int64_t ld, int size, int elements) {
    return p == nullptr ||
           (reinterpret_cast<uintptr_t>(p) % (uintptr_t)(size * elements) == 0 && ld % elements == 0);
}

inline bool aligned16(const void *p, int64_t ld, int size) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0);
}

template <class K, class A>
cudaError_t launch(K kernel, dim3 grid, dim3 block, const A &args, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace norm
}  // namespace sgemm
