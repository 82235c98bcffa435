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
// A warp adds the squares of its 512 to 1024 elements of a chunk in fp32 and its first lane
// adds that sum to a running one in 64 bits: 64-bit additions run at two a clock and SM here, so
// one a thread instead of one a warp was felt (12 MB in 28 tensors 22.9 us).  Where the fp32 sum
// has left the range in which it is exact to rounding (elements beyond 1e15, or all below 1e-12), the warp
// forms it again in 64 bits from the same registers.  CTAs' sums are stored in 64 bits and added in
// a fixed order by every CTA of the second launch: no atomics, the same bits every time.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "layer_math.cuh"
#include "layers.h"

namespace sgemm {
namespace clip {

constexpr int kThreads = 512;
constexpr int kCtas = 152 * 2;                          // of a launch at most: two an SM
constexpr int kAccesses = 4;                            // of 16 bytes, in flight a thread
constexpr int kChunk = kThreads * 16 * kAccesses;       // bytes

// One tensor of a launch.  Bytes are counted from the 16-byte boundary at or below its first
// element: it holds those from `lo` to `hi`.
struct Tensor {
    const char *x;   // that boundary
    char *y;         // the same place of the result
    int64_t hi;
    int first;       // chunks before it in this launch
    uint8_t type, lo, same;   // same: y's boundary is one too
};
// start[b]: the tensor that CTA b's first chunk is in (a search would be dependent reads of
// arguments that no cache holds yet).
template <int MOST>
struct Table {
    int count, chunks;   // tensors, chunks
    uint16_t start[kCtas + 1];
    Tensor t[MOST];
};
// a kernel's arguments may take 32764 bytes
constexpr int kMost = 1000;
static_assert(sizeof(Table<kMost>) <= 32700, "kernel arguments");

__host__ __device__ inline int first_chunk(int chunks, int cta, int ctas) {
    return (int)((int64_t)chunks * cta / ctas);
}

// This CTA's chunks, one after another, forward or backward: the chunk's tensor and where in
// it the chunk begins.
template <bool BACK, int MOST>
struct Walk {
    const Table<MOST> &table;
    int c, left, i;
    __device__ __forceinline__ explicit Walk(const Table<MOST> &t) : table(t) {
        const int c0 = first_chunk(t.chunks, blockIdx.x, gridDim.x);
        const int c1 = first_chunk(t.chunks, blockIdx.x + 1, gridDim.x);
        left = c1 - c0;
        c = BACK ? c1 - 1 : c0;
        i = t.start[blockIdx.x + (BACK ? 1 : 0)];
        if (left > 0) settle();
    }
    __device__ __forceinline__ void settle() {
        if (BACK) {
            while (table.t[i].first > c) --i;
        } else {
            while (i + 1 < table.count && table.t[i + 1].first <= c) ++i;
        }
    }
    __device__ __forceinline__ const Tensor &tensor() const { return table.t[i]; }
    __device__ __forceinline__ int64_t base() const {
        return (int64_t)(c - table.t[i].first) * kChunk;
    }
    __device__ __forceinline__ void next() {
        c += BACK ? -1 : 1;
        if (--left > 0) settle();
    }
};

// This thread's pieces of a chunk, as loaded; bytes that the tensor has not are 0.
struct Pieces {
    uint4 u[kAccesses];
    __device__ __forceinline__ void load(const Tensor &t, int64_t base) {
        const int64_t at = base + threadIdx.x * 16;
#pragma unroll
        for (int i = 0; i < kAccesses; ++i) {
            const int64_t b = at + i * kThreads * 16;
            const uint4 *p = reinterpret_cast<const uint4 *>(t.x + b);
            u[i] = make_uint4(0, 0, 0, 0);
            if (b >= t.lo && b + 16 <= t.hi)
                u[i] = __ldcg(p);
            else if (b < t.hi && b + 16 > t.lo)
                u[i] = part(t, b);
        }
    }
    // (every type's elements are made of whole 2-byte halves)
    __device__ __noinline__ static uint4 part(const Tensor &t, int64_t b) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 8; ++h)
            if (b + 2 * h >= t.lo && b + 2 * h < t.hi)
                w[h / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(t.x + b + 2 * h)
                            << (16 * (h % 2));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <class T>
__device__ __forceinline__ void values(uint4 u, float (&f)[16 / sizeof(T)]) {
    Raw<T, 16 / sizeof(T)> r;
    r.u = u;
    r.get(f);
}

// d summed over the warp in a fixed order, in each of its lanes.
__device__ __forceinline__ double warp_sum(double d) {
    if (!__any_sync(0xffffffffu, d != 0.0)) return 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    return d;
}

// The sum of squares of a thread's pieces in 64 bits.  (Not inlined: the registers it takes
// would leave the rest of the kernel spilling, 4.1 TB/s of bf16 instead of 6.6.)
template <class T>
__device__ __noinline__ double wide_squares(uint4 a, uint4 b, uint4 c, uint4 d) {
    const uint4 u[4] = {a, b, c, d};
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[16 / sizeof(T)];
        values<T>(u[i], f);
#pragma unroll
        for (int j = 0; j < 16 / (int)sizeof(T); ++j)
            if (f[j] != 0.f) s = fma((double)f[j], (double)f[j], s);   // (a NaN is not 0)
    }
    return s;
}

// The sum of squares of the warp's elements of a chunk.
template <class T>
__device__ __forceinline__ double chunk_squares(const Pieces &p) {
    constexpr int W = 16 / sizeof(T);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kAccesses; ++i) {
        float f[W];
        values<T>(p.u[i], f);
#pragma unroll
        for (int j = 0; j < W; ++j) s[j & 1] = fmaf(f[j], f[j], s[j & 1]);
    }
    float sum = s[0] + s[1];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // Below 2^-80 squares of elements may have lost their digits, from 2^100 on they may have
    // passed fp32's range.  (f16's squares, from 2^-48 to 2^32, do neither.)
    if constexpr (!std::is_same<T, __half>::value) {
        if (!(sum >= 0x1p-80f && sum < 0x1p100f)) {   // (the same in every lane)
            // (past a tensor's end there are zeros: fetching the 64-bit code for them was half of
            // a small list's time)
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < kAccesses; ++i) any |= p.u[i].x | p.u[i].y | p.u[i].z | p.u[i].w;
            if (!__any_sync(0xffffffffu, any != 0)) return 0.0;
            static_assert(kAccesses == 4, "the arguments below");
            return warp_sum(wide_squares<T>(p.u[0], p.u[1], p.u[2], p.u[3]));
        }
    }
    return (double)sum;
}

// partial[blockIdx.x] = the sum of squares of this CTA's chunks.  A chunk's loads are issued
// before the one before it is summed.
template <int MOST>
__global__ void __launch_bounds__(kThreads, 2)
squares_kernel(const __grid_constant__ Table<MOST> table, double *partial) {
    __shared__ double red[kThreads / 32];
    pdl_trigger();
    pdl_wait();
    double d = 0.0;
    const bool first = (threadIdx.x & 31) == 0;
    Walk<false, MOST> w(table);
    Pieces p, ahead;
    if (w.left > 0) ahead.load(w.tensor(), w.base());
    while (w.left > 0) {
        const int type = w.tensor().type;
        p = ahead;
        w.next();
        if (w.left > 0) ahead.load(w.tensor(), w.base());
        double s;
        switch (type) {
            case SGEMM_F32: s = chunk_squares<float>(p); break;
            case SGEMM_BF16: s = chunk_squares<__nv_bfloat16>(p); break;
            default: s = chunk_squares<__half>(p); break;
        }
        if (first) d += s;
    }
    if (first) red[threadIdx.x >> 5] = d;
    __syncthreads();
    if (threadIdx.x < 32) {
        const double s = warp_sum(threadIdx.x < kThreads / 32 ? red[threadIdx.x] : 0.0);
        if (threadIdx.x == 0) partial[blockIdx.x] = s;
    }
}

template <class T>
__device__ __forceinline__ void scale_chunk(const Pieces &p, const Tensor &t, int64_t base,
                                            float2 factor) {
    constexpr int W = 16 / sizeof(T);
    const int64_t first = base + threadIdx.x * 16;
#pragma unroll
    for (int i = 0; i < kAccesses; ++i) {
        const int64_t at = first + i * kThreads * 16;
        if (at >= t.hi) continue;
        float f[W];
        values<T>(p.u[i], f);
#pragma unroll
        for (int j = 0; j < W; ++j) f[j] = f[j] * factor.x * factor.y;
        if (t.same && at >= t.lo && at + 16 <= t.hi) {
            Raw<T, W> r;
            put<T, W>(reinterpret_cast<T *>(&r), f);
            __stcs(reinterpret_cast<uint4 *>(t.y + at), r.u);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int64_t b = at + j * (int)sizeof(T);
                if (b >= t.lo && b < t.hi) *reinterpret_cast<T *>(t.y + b) = from_f32<T>(f[j]);
            }
        }
    }
}

// The norm from all CTAs' sums (*norm, by the first CTA), and this CTA's chunks scaled.
template <int MOST>
__global__ void __launch_bounds__(kThreads, 2)
scale_kernel(const __grid_constant__ Table<MOST> table, const double *partial, int parts,
             float max_norm, float eps, float *norm) {
    __shared__ float2 shared_factor;
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x < 32) {
        constexpr int U = 10;   // in flight; a launch's sums of CTAs in one go
        double sum = 0.0;
        for (int i = threadIdx.x; i < parts; i += 32 * U) {
            double x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                x[u] = i + 32 * u < parts ? __ldcg(partial + i + 32 * u) : 0.0;
#pragma unroll
            for (int u = 0; u < U; ++u) sum += x[u];
        }
        const double n = sqrt(warp_sum(sum));
        if (threadIdx.x == 0) {
            if (norm != nullptr && blockIdx.x == 0) *norm = (float)n;
            // (nothing to scale where both are 0; no bound scales nothing, an infinite norm or not)
            const double d = n + (double)eps, bound = (double)max_norm;
            const double c = d == 0.0 || (isinf(bound) && isinf(d)) ? 1.0 : bound / d;
            // A factor that fp32 holds with few digits or not at all is applied in two steps, the
            // second a power of two; what the first one's product loses below fp32's normal range,
            // the second makes 0.  (Down to 2^-278, whose product with any element is 0.  A NaN
            // stays one.)
            const bool tiny = c < 0x1p-120, far = c < 0x1p-184;
            const double held = far ? c * 0x1p148 : tiny ? c * 0x1p64 : c;
            shared_factor = make_float2(c > 1.0 ? 1.f : (float)held,
                                        far ? 0x1p-148f : tiny ? 0x1p-64f : 1.f);
        }
    }
    Walk<true, MOST> w(table);
    Pieces p;
    if (w.left > 0) p.load(w.tensor(), w.base());
    __syncthreads();
    const float2 factor = shared_factor;
    auto changes = [&](const Tensor &t) { return !(factor.x == 1.f && t.y == t.x); };
    while (w.left > 0) {
        const Tensor &t = w.tensor();
        const int64_t base = w.base();
        if (changes(t)) {
            switch (t.type) {
                case SGEMM_F32: scale_chunk<float>(p, t, base, factor); break;
                case SGEMM_BF16: scale_chunk<__nv_bfloat16>(p, t, base, factor); break;
                default: scale_chunk<__half>(p, t, base, factor); break;
            }
        }
        w.next();
        if (w.left > 0 && changes(w.tensor())) p.load(w.tensor(), w.base());
    }
}

// ------------------------------------------------------------------ host side

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

int grid_of(int chunks) { return chunks < kCtas ? chunks : kCtas; }

// Tensors first .. of the list, as many as a table takes, without the empty ones; returns the
// next one's number, that of a tensor with elements or `count`: the empty ones behind a full
// table are passed over too, as a call for them alone would only clear the table.
template <int MOST>
int64_t fill(Table<MOST> &table, int64_t first, int64_t count, const int *types,
             const int64_t *sizes, const void *const *X, void *const *Y) {
    table.count = table.chunks = 0;
    int64_t i = first;
    for (; i < count && (table.count < MOST || sizes[i] == 0); ++i) {
        if (sizes[i] == 0) continue;
        Tensor &t = table.t[table.count];
        const uintptr_t x = reinterpret_cast<uintptr_t>(X[i]);
        const uintptr_t y = Y != nullptr ? reinterpret_cast<uintptr_t>(Y[i]) : x;
        const int off = (int)(x % 16);
        const int64_t hi = off + sizes[i] * dtype_size(types[i]), chunks = (hi + kChunk - 1) / kChunk;
        if (table.chunks + chunks > 0x7fffffff) {
            if (table.count == 0) return -1;
            break;
        }
        t.x = reinterpret_cast<const char *>(x - off);
        t.y = reinterpret_cast<char *>(y - off);
        t.hi = hi;
        t.first = table.chunks;
        t.type = (uint8_t)types[i];
        t.lo = (uint8_t)off;
        t.same = (y - off) % 16 == 0;
        table.chunks += (int)chunks;
        ++table.count;
    }
    const int ctas = grid_of(table.chunks);
    for (int b = 0, k = 0; b <= ctas && table.count > 0; ++b) {
        const int c = first_chunk(table.chunks, b, ctas);
        while (k + 1 < table.count && table.t[k + 1].first <= c) ++k;
        table.start[b] = (uint16_t)k;
    }
    return i;
}

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
        if (table.chunks == 0) break;   // (a list of empty tensors)
        const cudaError_t e = launch(squares_kernel<MOST>, grid_of(table.chunks), s, table,
                                     partial + parts);
        if (e != cudaSuccess) return e;
        parts += grid_of(table.chunks);
        ++tables;
    }
    const double *sums = partial;
    if (Y == nullptr || parts == 0) {
        table.count = table.chunks = 0;
        table.start[0] = table.start[1] = 0;
        return launch(scale_kernel<MOST>, 1, s, table, sums, parts, max_norm, eps, norm);
    }
    i = 0;
    while (i < count) {
        const bool first = i == 0;
        if (tables == 1) i = count;   // it still holds the list
        else i = fill(table, i, count, types, sizes, X, Y);
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
