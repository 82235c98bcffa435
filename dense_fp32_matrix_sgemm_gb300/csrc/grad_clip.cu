// The norm of all elements of a list of tensors, and the tensors scaled so that it is at
// most max_norm:
//
//   norm = (sum over tensors and elements of x^2)^(1/2)
//   y = x min(1, max_norm / (norm + eps))
//
// HBM bounds it (two operations an element): every element is read for the sum and, once that
// is known, read again and written, in two launches for the whole list, whatever the number
// of tensors; the tensors' addresses and sizes travel as the launches' own arguments, so no
// copy precedes them and a captured call holds them.  The list is cut into chunks of 32 KB
// that never cross a tensor; a CTA takes a run of consecutive chunks, forward in the sum and
// backward in the scaling, so that what each CTA read last, which L2 (129 MB) still holds, is
// read first.
// A thread adds the squares of 16 to 64 elements in fp32 and adds that sum to a running sum
// in 64 bits (one such addition for all of them).  Where the fp32 sum has left the range
// in which it is exact to rounding (elements beyond 1e15, or all below 1e-12), the thread forms it
// again in 64 bits from the same registers.  CTAs' sums are stored in 64 bits and added in
// a fixed order by every CTA of the second launch: no atomics, the same bits every time.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "layer_math.cuh"
#include "layers.h"

namespace sgemm {
namespace clip {

constexpr int kThreads = 256;
constexpr int kAccesses = 8;                            // of 16 bytes, in flight a thread
constexpr int kChunk = kThreads * 16 * kAccesses;       // bytes

// One tensor of a launch.  Elements are counted from the 16-byte boundary at or below its
// first one: it holds those from `shift` to `end`.
struct Tensor {
    const char *x;   // that boundary
    char *y;         // the same place of the result: x + anything; null: not scaled
    int64_t end;
    int first;       // chunks before it in this launch
    uint8_t type, shift, same;   // same: y's boundary is one too
};
template <int MOST>
struct Table {
    int count, chunks;   // tensors, chunks
    Tensor t[MOST];
};
// a kernel's arguments may take 32764 bytes
constexpr int kMost = 1000;
static_assert(sizeof(Table<kMost>) <= 32700, "kernel arguments");

// The tensor of the table that chunk c is in.
template <int MOST>
__device__ __forceinline__ int tensor_of(const Table<MOST> &table, int c) {
    int lo = 0, hi = table.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table.t[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// f(tensor, first element of the chunk) for this CTA's chunks, forward or backward.
template <bool BACK, int MOST, class F>
__device__ __forceinline__ void for_chunks(const Table<MOST> &table, F f) {
    const int c0 = (int)((int64_t)table.chunks * blockIdx.x / gridDim.x);
    const int c1 = (int)((int64_t)table.chunks * (blockIdx.x + 1) / gridDim.x);
    if (c0 >= c1) return;
    int i = tensor_of(table, BACK ? c1 - 1 : c0);
    for (int k = 0; k < c1 - c0; ++k) {
        const int c = BACK ? c1 - 1 - k : c0 + k;
        if (BACK) {
            while (table.t[i].first > c) --i;
        } else {
            while (i + 1 < table.count && table.t[i + 1].first <= c) ++i;
        }
        const Tensor &t = table.t[i];
        f(t, (int64_t)(c - t.first) * (t.type == SGEMM_F32 ? kChunk / 4 : kChunk / 2));
    }
}

// W elements from `at` on, those that the tensor has (others are 0).
template <class T>
struct Piece {
    static constexpr int W = 16 / sizeof(T);
    Raw<T, W> raw;
    __device__ __forceinline__ void load(const Tensor &t, int64_t at) {
        const T *x = reinterpret_cast<const T *>(t.x);
        if (at >= t.shift && at + W <= t.end) {
            raw.u = __ldcg(reinterpret_cast<const uint4 *>(x + at));
        } else {
            float f[W];
#pragma unroll
            for (int j = 0; j < W; ++j)
                f[j] = at + j >= t.shift && at + j < t.end ? to_f32(x[at + j]) : 0.f;
            if constexpr (W == 4)
                raw.u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                                   __float_as_uint(f[2]), __float_as_uint(f[3]));
            else
                raw.u = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                                   pack2<T>(f[6], f[7]));
        }
    }
};

template <class T>
__device__ __forceinline__ double chunk_squares(const Tensor &t, int64_t base) {
    using P = Piece<T>;
    P p[kAccesses];
#pragma unroll
    for (int i = 0; i < kAccesses; ++i) p[i].load(t, base + (i * kThreads + threadIdx.x) * P::W);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kAccesses; ++i) {
        float f[P::W];
        p[i].raw.get(f);
#pragma unroll
        for (int j = 0; j < P::W; ++j) s[j & 1] = fmaf(f[j], f[j], s[j & 1]);
    }
    const float sum = s[0] + s[1];
    // Below 2^-80 squares of elements may have lost their digits, from 2^100 on they may have
    // passed fp32's range.  (f16's squares, from 2^-48 to 2^32, do neither.)
    if constexpr (!std::is_same<T, __half>::value) {
        if (!(sum >= 0x1p-80f && sum < 0x1p100f)) {
            double d = 0.0;
#pragma unroll
            for (int i = 0; i < kAccesses; ++i) {
                float f[P::W];
                p[i].raw.get(f);
#pragma unroll
                for (int j = 0; j < P::W; ++j)
                    if (f[j] != 0.f) d = fma((double)f[j], (double)f[j], d);   // (a NaN is not 0)
            }
            return d;
        }
    }
    return (double)sum;
}

// d summed over the CTA, in each of its threads; in a fixed order.
__device__ __forceinline__ double block_sum(double d, double *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = d;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    return s;
}

// partial[blockIdx.x] = the sum of squares of this CTA's chunks.
template <int MOST>
__global__ void __launch_bounds__(kThreads, 4)
squares_kernel(const __grid_constant__ Table<MOST> table, double *partial) {
    __shared__ double red[kThreads / 32];
    pdl_trigger();
    pdl_wait();
    double d = 0.0;
    for_chunks<false>(table, [&](const Tensor &t, int64_t base) {
        switch (t.type) {
            case SGEMM_F32: d += chunk_squares<float>(t, base); break;
            case SGEMM_BF16: d += chunk_squares<__nv_bfloat16>(t, base); break;
            default: d += chunk_squares<__half>(t, base); break;
        }
    });
    const double s = block_sum(d, red);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

template <class T>
__device__ __forceinline__ void scale_chunk(const Tensor &t, int64_t base, float coef,
                                            float rest) {
    using P = Piece<T>;
    P p[kAccesses];
#pragma unroll
    for (int i = 0; i < kAccesses; ++i) p[i].load(t, base + (i * kThreads + threadIdx.x) * P::W);
    T *const y = reinterpret_cast<T *>(t.y);
#pragma unroll
    for (int i = 0; i < kAccesses; ++i) {
        const int64_t at = base + (i * kThreads + threadIdx.x) * P::W;
        if (at >= t.end) continue;
        float f[P::W];
        p[i].raw.get(f);
#pragma unroll
        for (int j = 0; j < P::W; ++j) f[j] = f[j] * coef * rest;
        if (t.same && at >= t.shift && at + P::W <= t.end) {
            put<T, P::W>(y + at, f);
        } else {
#pragma unroll
            for (int j = 0; j < P::W; ++j)
                if (at + j >= t.shift && at + j < t.end) y[at + j] = from_f32<T>(f[j]);
        }
    }
}

// The norm from all CTAs' sums (*norm, by the first CTA), and this CTA's chunks scaled.
template <int MOST>
__global__ void __launch_bounds__(kThreads, 4)
scale_kernel(const __grid_constant__ Table<MOST> table, const double *partial, int parts,
             float max_norm, float eps, float *norm) {
    __shared__ double red[kThreads / 32];
    pdl_trigger();
    pdl_wait();
    double d = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) d += __ldcg(partial + i);
    const double n = sqrt(block_sum(d, red));
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    const double c = (double)max_norm / (n + (double)eps);
    // (a NaN stays one; a factor that fp32 holds with few digits, for norms beyond 1e36 times
    // max_norm, is applied in two steps)
    const bool tiny = c < 0x1p-120;
    const float coef = c > 1.0 ? 1.f : (float)(tiny ? c * 0x1p64 : c);
    const float rest = tiny ? 0x1p-64f : 1.f;
    for_chunks<true>(table, [&](const Tensor &t, int64_t base) {
        if (coef == 1.f && t.y == t.x) return;   // in place: unchanged
        switch (t.type) {
            case SGEMM_F32: scale_chunk<float>(t, base, coef, rest); break;
            case SGEMM_BF16: scale_chunk<__nv_bfloat16>(t, base, coef, rest); break;
            default: scale_chunk<__half>(t, base, coef, rest); break;
        }
    });
}

// ------------------------------------------------------------------ host side

constexpr int kCtas = 152 * 4;   // of a launch at most

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), int grid, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tensors first .. of the list, as many as a table takes, without the empty ones; returns the
// next one's number.
template <int MOST>
int64_t fill(Table<MOST> &table, int64_t first, int64_t count, const int *types,
             const int64_t *sizes, const void *const *X, void *const *Y) {
    table.count = table.chunks = 0;
    int64_t i = first;
    for (; i < count && table.count < MOST; ++i) {
        if (sizes[i] == 0) continue;
        const int size = dtype_size(types[i]), per = kChunk / size;
        Tensor &t = table.t[table.count];
        const uintptr_t x = reinterpret_cast<uintptr_t>(X[i]);
        const uintptr_t y = Y != nullptr ? reinterpret_cast<uintptr_t>(Y[i]) : x;
        const int off = (int)(x % 16);
        const int64_t end = sizes[i] + off / size, chunks = (end + per - 1) / per;
        if (table.chunks + chunks > 0x7fffffff) {
            if (table.count == 0) return -1;
            break;
        }
        t.x = reinterpret_cast<const char *>(x - off);
        t.y = reinterpret_cast<char *>(y - off);
        t.end = end;
        t.first = table.chunks;
        t.type = (uint8_t)types[i];
        t.shift = (uint8_t)(off / size);
        t.same = (y - off) % 16 == 0;
        table.chunks += (int)chunks;
        ++table.count;
    }
    return i;
}

int grid_of(int chunks) { return chunks < kCtas ? chunks : kCtas; }

template <int MOST>
cudaError_t run(int64_t count, const int *types, const int64_t *sizes, const void *const *X,
                void *const *Y, float max_norm, float eps, float *norm, double *partial,
                cudaStream_t s) {
    Table<MOST> table;
    int parts = 0, tables = 0;
    int64_t i = 0;
    while (i < count) {
        i = fill(table, i, count, types, sizes, X, Y);
        if (i < 0) return cudaErrorInvalidValue;
        if (table.chunks == 0) break;
        const cudaError_t e = launch(squares_kernel<MOST>, grid_of(table.chunks), s, table,
                                     partial + parts);
        if (e != cudaSuccess) return e;
        parts += grid_of(table.chunks);
        ++tables;
    }
    const double *sums = partial;
    if (Y == nullptr || parts == 0) {
        table.count = table.chunks = 0;
        return launch(scale_kernel<MOST>, 1, s, table, sums, parts, max_norm, eps, norm);
    }
    i = 0;
    while (i < count) {
        const bool first = i == 0;
        if (tables == 1) i = count;   // it still holds the list
        else i = fill(table, i, count, types, sizes, X, Y);
        if (table.chunks == 0) break;
        const cudaError_t e = launch(scale_kernel<MOST>, grid_of(table.chunks), s, table, sums,
                                     parts, max_norm, eps, first ? norm : (float *)nullptr);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace clip

// CTAs' sums of as many launches as the list may take.
size_t grad_clip_bytes(int64_t count, const int *types, const int64_t *sizes) {
    int64_t launches = 1, tensors = 0, chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] <= 0) continue;
        const int per = clip::kChunk / dtype_size(types[i]);
        const int64_t c = sizes[i] / per + 2;
        if (tensors == clip::kMost || chunks + c > 0x7fffffff) {
            ++launches;
            tensors = chunks = 0;
        }
        ++tensors;
        chunks += c;
    }
    return (size_t)launches * clip::kCtas * sizeof(double);
}

cudaError_t launch_grad_clip(int64_t count, const int *types, const int64_t *sizes,
                             const void *const *X, void *const *Y, float max_norm, float eps,
                             float *norm, double *partial, cudaStream_t s) {
    // the smallest table that holds the list: a launch copies all of its arguments
    if (count <= 32)
        return clip::run<32>(count, types, sizes, X, Y, max_norm, eps, norm, partial, s);
    if (count <= 256)
        return clip::run<256>(count, types, sizes, X, Y, max_norm, eps, norm, partial, s);
    return clip::run<clip::kMost>(count, types, sizes, X, Y, max_norm, eps, norm, partial, s);
}

}  // namespace sgemm
