// Root-mean-square norm with the residual's addition, in the input's type or
// as 8-bit rows with a scale, its gradients, and the row quantiser.
//
//   s = x + r,  rstd = (mean s^2 + eps)^(-1/2),  y = s rstd w
//   g = dy w,   dx = ds + rstd (g - s rstd^2 mean(g s)),  dw = sum_rows dy s rstd
//
// HBM bounds all of them: a few operations per element that is read once and
// written once.  So a row is read once, in 16-byte accesses that are all
// issued before the first use, held in registers (fp32) by the threads of one
// row group, reduced once across the group, and written from the registers.
// The 8-bit output needs the row's largest |y| besides its sum of squares; as
// |y| = |s w| rstd, both reductions run at once on (sum s^2, max |s w|), with
// one barrier instead of two.
// A row group is tpr threads (a multiple of 32, up to 1024) times NV accesses
// of W elements; groups narrower than a CTA share it (blockDim.y of them).
// Rows wider than that are read twice, the second time from L2 (the *_wide
// kernels); bases or rows that are not 16-byte aligned take W = 1.
// Measured (bf16, of 6.79 TB/s copied): 8192 x 8192 with a residual 79.1 us, 6.79
// TB/s; 8192 x 8192 quantised 32.6 us, 6.2 TB/s; gradients of 8192 x 4096 47.8 us,
// 5.6 TB/s, of which the weight's partial sums and their pass are 4.5; one row of
// 4096 in 8 bits 6 us a call, which is the call's own time.
// The weight's gradient sums over rows: every group walks rows with the
// stride of the grid and keeps its columns' sums in registers, the CTAs' sums
// go to the workspace, and one more pass adds them in a fixed order.
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
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) p[i] = to_e4m3(y[i]);
    }
}

struct RowArgs {
    const void *X, *R, *w;
    void *S, *Y;
    int64_t ldx, ldr, lds, ldy, rows;
    float *q_scale, *rstd;
    float eps;
    int D;
};

// NORM: the norm (else y = x: the row quantiser).  QUANT: 8-bit output.
template <class T, int W, int NV, int MAXT, bool NORM, bool QUANT>
__global__ void __launch_bounds__(MAXT) row_kernel(const RowArgs a) {
    __shared__ float2 red[32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const T *x = static_cast<const T *>(a.X) + row * a.ldx;
    const T *r = static_cast<const T *>(a.R) + row * a.ldr;
    const T *w = static_cast<const T *>(a.w);
    Raw<T, W> vx[NV], vr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * W;
        const bool in = live && c < a.D;
        vx[i] = load_or_zero<T, W>(x + c, in);
        if (NORM && a.R != nullptr) vr[i] = load_or_zero<T, W>(r + c, in);
    }
    float s[NV][W];
    float sum = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * W;
        vx[i].get(s[i]);
        if (NORM && a.R != nullptr) {
            float r[W];
            vr[i].get(r);
#pragma unroll
            for (int j = 0; j < W; ++j) s[i][j] += r[j];
        }
        if constexpr (NORM) {
            if (a.S != nullptr && live && c < a.D)
                put<T, W>(static_cast<T *>(a.S) + row * a.lds + c, s[i]);
            float fw[W];
            load_or_zero<T, W>(w + c, c < a.D).get(fw);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                sum = fmaf(s[i][j], s[i][j], sum);
                s[i][j] *= fw[j];
            }
        }
        if constexpr (QUANT) {
#pragma unroll
            for (int j = 0; j < W; ++j) top = max_nan(top, fabsf(s[i][j]));
        }
    }
    const float2 t = group_reduce(sum, top, red);
    float mul = 1.f;
    if constexpr (NORM) {
        mul = 1.f / sqrtf(t.x / (float)max(a.D, 1) + a.eps);   // (no elements: a mean of 0)
        if (a.rstd != nullptr && live && threadIdx.x == 0) a.rstd[row] = mul;
    }
    if constexpr (QUANT) {
        const float amax = max_nan(t.y * mul, kAmaxFloor);
        if (live && threadIdx.x == 0) a.q_scale[row] = amax / kE4m3Max;
        const float inv = kE4m3Max / amax;
        uint8_t *q = static_cast<uint8_t *>(a.Y) + row * a.ldy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * W;
            if (!live || c >= a.D) continue;
            float y[W];
#pragma unroll
            for (int j = 0; j < W; ++j) y[j] = (NORM ? s[i][j] * mul : s[i][j]) * inv;
            store_codes<W>(q + c, y);
        }
    } else {
        T *out = static_cast<T *>(a.Y) + row * a.ldy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * W;
            if (!live || c >= a.D) continue;
            float y[W];
#pragma unroll
            for (int j = 0; j < W; ++j) y[j] = s[i][j] * mul;
            put<T, W>(out + c, y);
        }
    }
}

// Rows wider than a group's registers: one CTA a row, read again for the
// output.  S may be X or R: it is written in the second pass, each element
// after the same thread has read it.
template <class T, bool NORM, bool QUANT>
__global__ void __launch_bounds__(kMaxThreads) row_wide_kernel(const RowArgs a) {
    __shared__ float2 red[32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.X) + row * a.ldx;
    const T *r = a.R != nullptr ? static_cast<const T *>(a.R) + row * a.ldr : nullptr;
    const T *w = static_cast<const T *>(a.w);
    float sum = 0.f, top = 0.f;
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        float s = to_f32(x[c]);
        if (NORM) {
            if (r != nullptr) s += to_f32(r[c]);
            sum = fmaf(s, s, sum);
            s *= to_f32(w[c]);
        }
        top = max_nan(top, fabsf(s));
    }
    const float2 t = group_reduce(sum, top, red);
    float mul = 1.f;
    if constexpr (NORM) {
        mul = 1.f / sqrtf(t.x / (float)max(a.D, 1) + a.eps);   // (no elements: a mean of 0)
        if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = mul;
    }
    float inv = 1.f;
    if constexpr (QUANT) {
        const float amax = max_nan(t.y * mul, kAmaxFloor);
        if (threadIdx.x == 0) a.q_scale[row] = amax / kE4m3Max;
        inv = kE4m3Max / amax;
    }
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        float s = to_f32(x[c]);
        if (NORM) {
            if (r != nullptr) s += to_f32(r[c]);
            if (a.S != nullptr) static_cast<T *>(a.S)[row * a.lds + c] = from_f32<T>(s);
            s *= to_f32(w[c]);
        }
        const float y = NORM ? s * mul : s;
        if constexpr (QUANT)
            static_cast<uint8_t *>(a.Y)[row * a.ldy + c] = to_e4m3(y * inv);
        else
            static_cast<T *>(a.Y)[row * a.ldy + c] = from_f32<T>(y);
    }
}

struct GradArgs {
    const void *dY, *S, *w, *dS;
    void *dX;
    const float *rstd;
    float *partial;
    int64_t lddy, lds, ldds, lddx, rows;
    int D;
};

template <class T, int W, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) grad_kernel(const GradArgs a) {
    __shared__ float2 red[2][32];
    pdl_trigger();
    pdl_wait();
    const int64_t group = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t groups = (int64_t)gridDim.x * blockDim.y;
    Raw<T, W> vw[NV];
    float dw[NV][W];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * W;
        vw[i] = load_or_zero<T, W>(static_cast<const T *>(a.w) + c, c < a.D);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[i][j] = 0.f;
    }
    // every group of the CTA takes as many turns as its first one (barriers)
    const int64_t first = (int64_t)blockIdx.x * blockDim.y;
    const int turns = first < a.rows ? (int)((a.rows - 1 - first) / groups) + 1 : 0;
    // the next row's loads are issued before this row's sums where registers
    // allow it (CTAs of up to 512 threads)
    constexpr bool AHEAD = MAXT <= 512;
    Raw<T, W> ny[NV], ns[NV], nd[NV];
    float nr = 0.f;
    auto load_ds = [&](int64_t row, int c) {
        return load_or_zero<T, W>(static_cast<const T *>(a.dS) + row * a.ldds + c,
                                  row < a.rows && c < a.D && a.dS != nullptr);
    };
    auto load_row = [&](int64_t row) {
        const bool live = row < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * W;
            const bool in = live && c < a.D;
            ny[i] = load_or_zero<T, W>(static_cast<const T *>(a.dY) + row * a.lddy + c, in);
            ns[i] = load_or_zero<T, W>(static_cast<const T *>(a.S) + row * a.lds + c, in);
            if (AHEAD) nd[i] = load_ds(row, c);
        }
        nr = live ? a.rstd[row] : 0.f;
    };
    // where they do not, the next row is brought to L2 in the meantime, a lane a
    // 128-byte line (2048 x 16384 bf16 without dS: 88 -> 73 us), and dS is read only
    // when dX is formed, which leaves fewer registers to spill (70; now 66, with dS 75)
    auto prefetch_row = [&](int64_t row) {
        constexpr int LANES = W > 1 ? 128 / (W * (int)sizeof(T)) : 32;
        if (row >= a.rows || threadIdx.x % LANES != 0) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * W;
            if (c >= a.D) continue;
            prefetch_l2(static_cast<const T *>(a.dY) + row * a.lddy + c);
            prefetch_l2(static_cast<const T *>(a.S) + row * a.lds + c);
            if (a.dS != nullptr) prefetch_l2(static_cast<const T *>(a.dS) + row * a.ldds + c);
        }
    };
    if (AHEAD && turns > 0) load_row(group);
    for (int t = 0; t < turns; ++t) {
        const int64_t row = group + t * groups;
        const bool live = row < a.rows;
        if (!AHEAD) {
            load_row(row);
            if (t + 1 < turns) prefetch_row(row + groups);
        }
        Raw<T, W> vy[NV], vs[NV], vd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            vy[i] = ny[i];
            vs[i] = ns[i];
            if (AHEAD) vd[i] = nd[i];
        }
        const float rstd = nr;
        if (AHEAD && t + 1 < turns) load_row(row + groups);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float dy[W], s[W], w[W];
            vy[i].get(dy);
            vs[i].get(s);
            vw[i].get(w);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float ys = dy[j] * s[j];
                sum = fmaf(ys, w[j], sum);
                dw[i][j] = fmaf(ys, rstd, dw[i][j]);
            }
        }
        // two buffers: a warp may reach the next turn's while another still
        // reads this one's, not the one after (that takes the next barrier)
        // (the mean by a division: a rounded 1 / D would double its error)
        const float k = group_reduce(sum, 0.f, red[t & 1]).x / (float)a.D * rstd * rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * W;
            if (!live || c >= a.D) continue;
            float dy[W], s[W], w[W], ds[W], dx[W];
            vy[i].get(dy);
            vs[i].get(s);
            vw[i].get(w);
            (AHEAD ? vd[i] : load_ds(row, c)).get(ds);
#pragma unroll
            for (int j = 0; j < W; ++j)
                dx[j] = fmaf(rstd, fmaf(-k, s[j], dy[j] * w[j]), ds[j]);
            put<T, W>(static_cast<T *>(a.dX) + row * a.lddx + c, dx);
        }
    }
    if (a.partial == nullptr) return;
    // one row of partial sums a CTA: its groups' sums are added in their order
    // (groups share a CTA only up to 512 threads)
    __shared__ float sums[512 * NV * W];
    const int width = blockDim.x * NV * W;
    if (blockDim.y > 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j)
                sums[threadIdx.y * width + (i * W + j) * blockDim.x + threadIdx.x] = dw[i][j];
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 1; y < (int)blockDim.y; ++y)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    dw[i][j] += sums[y * width + (i * W + j) * blockDim.x + threadIdx.x];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * W;
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (c + j < a.D) a.partial[(int64_t)blockIdx.x * a.D + c + j] = dw[i][j];
    }
}

// Rows wider than a group's registers: the CTA reads each of its rows twice
// and keeps its columns' sums of dw in its own row of the workspace.
template <class T>
__global__ void __launch_bounds__(kMaxThreads) grad_wide_kernel(const GradArgs a) {
    __shared__ float2 red[2][32];
    pdl_trigger();
    pdl_wait();
    const T *w = static_cast<const T *>(a.w);
    float *part = a.partial != nullptr ? a.partial + (int64_t)blockIdx.x * a.D : nullptr;
    int t = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++t) {
        const T *dy = static_cast<const T *>(a.dY) + row * a.lddy;
        const T *s = static_cast<const T *>(a.S) + row * a.lds;
        const float rstd = a.rstd[row];
        float sum = 0.f;
        for (int c = threadIdx.x; c < a.D; c += blockDim.x)
            sum = fmaf(to_f32(dy[c]) * to_f32(w[c]), to_f32(s[c]), sum);
        const float k = group_reduce(sum, 0.f, red[t & 1]).x / (float)a.D * rstd * rstd;
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            const float y = to_f32(dy[c]), v = to_f32(s[c]);
            float dx = rstd * fmaf(-k, v, y * to_f32(w[c]));
            if (a.dS != nullptr) dx += to_f32(static_cast<const T *>(a.dS)[row * a.ldds + c]);
            if (part != nullptr) part[c] = fmaf(y * rstd, v, t > 0 ? part[c] : 0.f);
            static_cast<T *>(a.dX)[row * a.lddx + c] = from_f32<T>(dx);
        }
    }
}

// ------------------------------------------------------------------ host side

// Threads of a row group and groups of a CTA for n accesses a row, nv a
// thread; tpr 0 when the row does not fit a group.
struct Shape {
    int tpr, groups;
};
Shape shape_for(int64_t n, int nv) {
    const int64_t per = (n + nv - 1) / nv;
    if (per > kMaxThreads) return {0, 0};
    Shape s;
    s.tpr = per <= 32 ? 32 : (int)((per + 31) / 32 * 32);
    s.groups = s.tpr >= 256 ? 1 : 256 / s.tpr;
    return s;
}

bool aligned16(const void *p, int64_t ld, int size) {
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

// CTAs of up to 512 threads get the registers that hold a row without
// spilling; only the widest rows need the 1024-thread form (64 registers).
template <class T, int W, int NV, bool NORM, bool QUANT>
cudaError_t launch_row(const RowArgs &a, Shape sh, cudaStream_t s) {
    const dim3 grid((unsigned)((a.rows + sh.groups - 1) / sh.groups));
    const dim3 block((unsigned)sh.tpr, (unsigned)sh.groups);
    if (sh.tpr <= 512) return launch(row_kernel<T, W, NV, 512, NORM, QUANT>, grid, block, a, s);
    return launch(row_kernel<T, W, NV, kMaxThreads, NORM, QUANT>, grid, block, a, s);
}

template <class T, bool NORM, bool QUANT>
cudaError_t row_dispatch(const RowArgs &a, bool vec, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    if (vec) {
        const int64_t n = a.D / W;
        Shape sh = shape_for(n, 1);
        // few rows: as many threads as possible on each, for its latency
        if (sh.tpr > 0 && a.rows <= 304) return launch_row<T, W, 1, NORM, QUANT>(a, sh, s);
        sh = shape_for(n, 4);
        if (sh.tpr > 0) return launch_row<T, W, 4, NORM, QUANT>(a, sh, s);
    } else {
        const Shape sh = shape_for(a.D, 8);
        if (sh.tpr > 0) return launch_row<T, 1, 8, NORM, QUANT>(a, sh, s);
    }
    return launch(row_wide_kernel<T, NORM, QUANT>, dim3((unsigned)a.rows), dim3(kMaxThreads), a, s);
}

template <bool NORM, bool QUANT>
cudaError_t row_types(int type, const RowArgs &a, cudaStream_t s) {
    const int size = dtype_size(type), w = 16 / size;
    const bool vec = a.D % w == 0 && aligned16(a.X, a.ldx, size) && aligned16(a.R, a.ldr, size) &&
                     aligned16(a.w, 0, size) && aligned16(a.S, a.lds, size) &&
                     (QUANT ? reinterpret_cast<uintptr_t>(a.Y) % 8 == 0 && a.ldy % 8 == 0
                            : aligned16(a.Y, a.ldy, size));
    if (type == SGEMM_F32) return row_dispatch<float, NORM, QUANT>(a, vec, s);
    if (type == SGEMM_BF16) return row_dispatch<__nv_bfloat16, NORM, QUANT>(a, vec, s);
    return row_dispatch<__half, NORM, QUANT>(a, vec, s);
}

// The backward pass's row groups: as many CTAs as the SMs hold at once, at
// most one group a row.
struct GradShape {
    int w, nv;      // elements an access, accesses a thread; nv 0: the wide kernel
    Shape sh;
    int ctas;
};
GradShape grad_shape(int type, int64_t rows, int64_t D, bool vec) {
    GradShape g;
    g.w = vec ? 16 / dtype_size(type) : 1;
    const int64_t n = (D + g.w - 1) / g.w;
    g.nv = vec ? 2 : 8;
    g.sh = shape_for(n, g.nv);
    if (g.sh.tpr == 0) {
        g.nv = 0;
        g.sh = {kMaxThreads, 1};
    }
    // one CTA of 512 threads an SM has half the partial sums to write and add of two
    // of 256 (8192 x 4096 bf16: 48.8 -> 47.1 us); its groups wait for one another
    // (4096 x 1024: 7.9 -> 8.3), so only where each takes eight turns or more
    if (g.sh.tpr <= 256 && rows >= 152 * 8 * (512 / g.sh.tpr)) g.sh.groups = 512 / g.sh.tpr;
    const int64_t need = (rows + g.sh.groups - 1) / g.sh.groups;
    // up to 128 registers a thread: 512 threads an SM, the row of each group and
    // its next one in flight
    const int threads = g.sh.tpr * g.sh.groups;
    const int per_sm = threads > 512 ? 1 : 512 / threads;
    const int64_t most = (int64_t)152 * per_sm;
    g.ctas = (int)(need < most ? need : most);
    return g;
}

template <class T>
cudaError_t grad_dispatch(const GradArgs &a, const GradShape &g, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    const dim3 grid((unsigned)g.ctas), block((unsigned)g.sh.tpr, (unsigned)g.sh.groups);
    if (g.nv == 0) return launch(grad_wide_kernel<T>, grid, block, a, s);
    if (g.w == 1)
        return g.sh.tpr <= 512 ? launch(grad_kernel<T, 1, 8, 512>, grid, block, a, s)
                               : launch(grad_kernel<T, 1, 8, kMaxThreads>, grid, block, a, s);
    return g.sh.tpr <= 512 ? launch(grad_kernel<T, W, 2, 512>, grid, block, a, s)
                           : launch(grad_kernel<T, W, 2, kMaxThreads>, grid, block, a, s);
}

}  // namespace norm

cudaError_t launch_add_rmsnorm(int type, int64_t rows, int64_t D, const void *X, int64_t ldx,
                               const void *R, int64_t ldr, const void *w, float eps, void *S,
                               int64_t lds, void *Y, int64_t ldy, float *q_scale, float *rstd,
                               cudaStream_t s) {
    const norm::RowArgs a = {X, R, w, S, Y, ldx, ldr, lds, ldy, rows, q_scale, rstd, eps, (int)D};
    return q_scale != nullptr ? norm::row_types<true, true>(type, a, s)
                              : norm::row_types<true, false>(type, a, s);
}

cudaError_t launch_quantize_rows(int type, int64_t rows, int64_t D, const void *X, int64_t ldx,
                                 void *Q, int64_t ldq, float *scale, cudaStream_t s) {
    const norm::RowArgs a = {X,   nullptr, nullptr, nullptr, Q,       ldx,    0,
                             0,   ldq,     rows,    scale,   nullptr, 0.f,    (int)D};
    return norm::row_types<false, true>(type, a, s);
}

// Rows of partial sums, the larger of the aligned and the unaligned plan (the
// caller's pointers decide which one runs).
int rmsnorm_backward_parts(int type, int64_t rows, int64_t D) {
    const norm::GradShape a = norm::grad_shape(type, rows, D, true);
    const norm::GradShape b = norm::grad_shape(type, rows, D, false);
    return a.ctas > b.ctas ? a.ctas : b.ctas;
}

cudaError_t launch_add_rmsnorm_backward(int type, int64_t rows, int64_t D, const void *dY,
                                        int64_t lddy, const void *S, int64_t lds,
                                        const float *rstd, const void *w, const void *dS,
                                        int64_t ldds, void *dX, int64_t lddx, void *dw,
                                        float *partial, cudaStream_t s) {
    const int size = dtype_size(type), width = 16 / size;
    const bool vec = D % width == 0 && norm::aligned16(dY, lddy, size) &&
                     norm::aligned16(S, lds, size) && norm::aligned16(w, 0, size) &&
                     norm::aligned16(dS, ldds, size) && norm::aligned16(dX, lddx, size);
    const norm::GradShape g = norm::grad_shape(type, rows, D, vec);
    const norm::GradArgs a = {dY,   S,   w,    dS,   dX,   rstd, dw != nullptr ? partial : nullptr,
                              lddy, lds, ldds, lddx, rows, (int)D};
    cudaError_t e = type == SGEMM_F32    ? norm::grad_dispatch<float>(a, g, s)
                    : type == SGEMM_BF16 ? norm::grad_dispatch<__nv_bfloat16>(a, g, s)
                                         : norm::grad_dispatch<__half>(a, g, s);
    if (e != cudaSuccess || dw == nullptr) return e;
    return launch_column_sum(type, partial, g.ctas, D, dw, 0, s);
}

}  // namespace sgemm
