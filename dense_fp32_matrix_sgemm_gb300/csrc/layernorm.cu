// Layer norm with the residual's addition, in the input's type or as 8-bit rows with a
// scale, and its gradients.
//
//   s = x + r,  m = mean s,  rstd = (mean (s - m)^2 + eps)^(-1/2),  n = (s - m) rstd,  y = n w + b
//   g = dy w,   dx = ds + rstd (g - mean g - n mean(g n)),  dw = sum_rows dy n,  db = sum_rows dy
//
// HBM bounds them as it bounds the root-mean-square norm, and the row groups, accesses and
// launches are norm.cu's: a row is read once into registers (fp32), and written from there.
// The statistics are formed from differences, not from sums of squares (which would lose a
// large mean's digits): first the mean, then the sums of s - m and of its square, where the
// first corrects both for the mean's own rounding.  That is two reductions across the group; the 8-bit output's largest |y| is
// a third, as the bias keeps it from being formed before rstd is known.
// The gradients' two row sums go through one reduction; the sums over rows of dw and db stay
// in registers over a group's rows, go to the workspace a row a CTA, and are added in a fixed
// order by one more pass.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "gemm_args.h"
#include "layer_math.cuh"
#include "layers.h"
#include "row_reduce.cuh"
#include "tc_issue.cuh"

namespace sgemm {
namespace norm {
namespace {

// Sums of a and b over the CTA's row group, the same in each of its threads.  red: 32 float2
// of shared memory that nothing else uses until two barriers later.
__device__ __forceinline__ float2 group_sum2(float a, float b, float2 *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    const int warps = blockDim.x >> 5;   // of one group
    if (warps == 1) return make_float2(a, b);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2 *mine = red + threadIdx.y * warps;
    if (lane == 0) mine[warp] = make_float2(a, b);
    __syncthreads();
    const float2 p = lane < warps ? mine[lane] : make_float2(0.f, 0.f);
    a = p.x;
    b = p.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return make_float2(a, b);
}

// Rows that start off a 16-byte boundary, all of a call's by as much in a row (an odd number of
// elements a row): `head` elements lead to the first boundary, `accesses` whole accesses follow,
// and the row's two ends (fewer than 32 elements) go one element a thread.  The last access
// that fits is left to the ends, as a vector's two accesses that hold its columns (load_moved)
// might pass the vector's end.
struct Shifted {
    int head, accesses;
    // the thread's element of the ends; D or more: none
    __device__ __forceinline__ int end(int W) const {
        const int x = threadIdx.x;
        return x < head ? x : accesses * W + x;
    }
};
template <class T, int W>
__device__ __forceinline__ Shifted shifted(const void *row, int D) {
    const int past = (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T) % W);
    if (past == 0) return {0, D / W};
    return {W - past, max(D / W - 1, 0)};
}

// Columns head + k W .. of a vector on a boundary, from its accesses k and k + 1.
template <class T, int W>
__device__ __forceinline__ Raw<T, W> load_moved(const T *p, int k, int head, bool in) {
    const Raw<T, W> lo = load_or_zero<T, W>(p + k * W, in);
    if (head == 0) return lo;   // (the same for a warp)
    const Raw<T, W> hi = load_or_zero<T, W>(p + (k + 1) * W, in);
    const uint32_t v[8] = {lo.u.x, lo.u.y, lo.u.z, lo.u.w, hi.u.x, hi.u.y, hi.u.z, hi.u.w};
    constexpr int WORD = 4 / (int)sizeof(T);   // elements
    const int words = head / WORD, bits = 16 * (head % WORD);
    uint32_t a[6], b[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) a[i] = words & 2 ? v[i + 2] : v[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) b[i] = words & 1 ? a[i + 1] : a[i];
    Raw<T, W> r;
    r.u = make_uint4(__funnelshift_r(b[0], b[1], bits), __funnelshift_r(b[1], b[2], bits),
                     __funnelshift_r(b[2], b[3], bits), __funnelshift_r(b[3], b[4], bits));
    return r;
}

struct LayerRowArgs {
    const void *X, *R, *w, *b;
    void *S, *Y;
    int64_t ldx, ldr, lds, ldy, rows;
    float *q_scale, *mean, *rstd;
    float eps;
    int D;
};

// QUANT: 8-bit output.  SHIFT: rows off the boundary (in 64 registers, MAXT 1024: moving the weights
// takes 93, which leaves an SM too few warps: 1280 x 6427 bf16 18.8 -> 14.7 us).
template <class T, int W, int NV, int MAXT, bool QUANT, bool SHIFT>
__global__ void __launch_bounds__(MAXT) layer_row_kernel(const LayerRowArgs a) {
    __shared__ float2 red[3][32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const T *x = static_cast<const T *>(a.X) + row * a.ldx;
    const T *r = static_cast<const T *>(a.R) + row * a.ldr;
    const T *w = static_cast<const T *>(a.w);
    const T *b = static_cast<const T *>(a.b);
    const Shifted at = SHIFT ? shifted<T, W>(x, a.D)  : Shifted{0, 0};
    const int end = SHIFT ? at.end(W) : a.D, limit = SHIFT ? at.head + at.accesses * W : a.D;
    const bool ends = end < a.D;
    auto column = [&](int i) {
        const int c = (i * blockDim.x + threadIdx.x) * W;
        return SHIFT ? c + at.head : c;
    };
    auto in = [&](int i) { return column(i) < limit; };
    Raw<T, W> vx[NV], vr[NV];
    Raw<T, 1> ex, er;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        vx[i] = load_or_zero<T, W>(x + column(i), live && in(i));
        if (a.R != nullptr) vr[i] = load_or_zero<T, W>(r + column(i), live && in(i));
    }
    if constexpr (SHIFT) {
        ex = load_or_zero<T, 1>(x + end, live && ends);
        er = load_or_zero<T, 1>(r + end, live && ends && a.R != nullptr);
    }
    float s[NV][W], e[1] = {0.f};
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        vx[i].get(s[i]);
        if (a.R != nullptr) {
            float r[W];
            vr[i].get(r);
#pragma unroll
            for (int j = 0; j < W; ++j) s[i][j] += r[j];
        }
        if (a.S != nullptr && live && in(i))
            put<T, W>(static_cast<T *>(a.S) + row * a.lds + column(i), s[i]);
#pragma unroll
        for (int j = 0; j < W; ++j) sum += s[i][j];
    }
    if constexpr (SHIFT) {
        e[0] = to_f32(ex.u) + to_f32(er.u);
        if (a.S != nullptr && live && ends)
            put<T, 1>(static_cast<T *>(a.S) + row * a.lds + end, e);
        sum += e[0];
    }
    const float width = (float)max(a.D, 1);   // (no elements: a mean and a variance of 0)
    const float first = group_sum2(sum, 0.f, red[0]).x / width;
    float off = 0.f, square = 0.f;
    auto differ = [&](float &s, bool in) {
        s = in ? s - first : 0.f;
        off += s;
        square = fmaf(s, s, square);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) differ(s[i][j], in(i));
    if constexpr (SHIFT) differ(e[0], ends);
    const float2 t = group_sum2(off, square, red[1]);
    const float shift = t.x / width;
    const float rstd = 1.f / sqrtf(max_nan(t.y / width - shift * shift, 0.f) + a.eps);
    if (live && threadIdx.x == 0) {
        if (a.mean != nullptr) a.mean[row] = isinf(first) ? first : first + shift;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float fw[W], fb[W];
        if constexpr (SHIFT) {
            load_moved<T, W>(w, (int)(i * blockDim.x + threadIdx.x), at.head, in(i)).get(fw);
            load_moved<T, W>(b, (int)(i * blockDim.x + threadIdx.x), at.head, in(i) && b != nullptr).get(fb);
        } else {
            load_or_zero<T, W>(w + column(i), in(i)).get(fw);
            load_or_zero<T, W>(b + column(i), in(i) && b != nullptr).get(fb);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            s[i][j] = fmaf((s[i][j] - shift) * rstd, fw[j], fb[j]);
            if (QUANT && in(i)) top = max_nan(top, fabsf(s[i][j]));
        }
        if (!QUANT && live && in(i))
            put<T, W>(static_cast<T *>(a.Y) + row * a.ldy + column(i), s[i]);
    }
    if (SHIFT && ends) {
        e[0] = fmaf((e[0] - shift) * rstd, to_f32(w[end]), b != nullptr ? to_f32(b[end]) : 0.f);
        top = max_nan(top, fabsf(e[0]));
        if (!QUANT && live) put<T, 1>(static_cast<T *>(a.Y) + row * a.ldy + end, e);
    }
    if constexpr (QUANT) {
        const float amax = max_nan(group_reduce(0.f, top, red[2]).y, kAmaxFloor);
        if (live && threadIdx.x == 0) a.q_scale[row] = amax / kE4m3Max;
        const float inv = kE4m3Max / amax;
        uint8_t *q = static_cast<uint8_t *>(a.Y) + row * a.ldy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!live || !in(i)) continue;
#pragma unroll
            for (int j = 0; j < W; ++j) s[i][j] *= inv;
            store_codes<W>(q + column(i), s[i]);
        }
        if (SHIFT && live && ends) q[end] = to_e4m3(e[0] * inv);
    }
}

// Rows wider than a group's registers: one CTA a row, read again (from L2) for each sum and
// for the output.  S may be X or R: it is written in the last pass, each element after the
// same thread has read it.
template <class T, bool QUANT>
__global__ void __launch_bounds__(kMaxThreads) layer_row_wide_kernel(const LayerRowArgs a) {
    __shared__ float2 red[3][32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.X) + row * a.ldx;
    const T *r = a.R != nullptr ? static_cast<const T *>(a.R) + row * a.ldr : nullptr;
    const T *w = static_cast<const T *>(a.w);
    const T *b = static_cast<const T *>(a.b);
    auto value = [&](int c) { return to_f32(x[c]) + (r != nullptr ? to_f32(r[c]) : 0.f); };
    float sum = 0.f;
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) sum += value(c);
    const float width = (float)max(a.D, 1);
    const float first = group_sum2(sum, 0.f, red[0]).x / width;
    float off = 0.f, square = 0.f;
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        const float s = value(c) - first;
        off += s;
        square = fmaf(s, s, square);
    }
    const float2 t = group_sum2(off, square, red[1]);
    const float shift = t.x / width;
    const float rstd = 1.f / sqrtf(max_nan(t.y / width - shift * shift, 0.f) + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean != nullptr) a.mean[row] = isinf(first) ? first : first + shift;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    auto output = [&](int c, float s) {
        return fmaf((s - first - shift) * rstd, to_f32(w[c]), b != nullptr ? to_f32(b[c]) : 0.f);
    };
    float inv = 1.f;
    if constexpr (QUANT) {
        float top = 0.f;
        for (int c = threadIdx.x; c < a.D; c += blockDim.x)
            top = max_nan(top, fabsf(output(c, value(c))));
        const float amax = max_nan(group_reduce(0.f, top, red[2]).y, kAmaxFloor);
        if (threadIdx.x == 0) a.q_scale[row] = amax / kE4m3Max;
        inv = kE4m3Max / amax;
    }
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        const float s = value(c);
        if (a.S != nullptr) static_cast<T *>(a.S)[row * a.lds + c] = from_f32<T>(s);
        const float y = output(c, s);
        if constexpr (QUANT)
            static_cast<uint8_t *>(a.Y)[row * a.ldy + c] = to_e4m3(y * inv);
        else
            static_cast<T *>(a.Y)[row * a.ldy + c] = from_f32<T>(y);
    }
}

struct LayerGradArgs {
    const void *dY, *S, *w, *dS;
    void *dX;
    const float *mean, *rstd;
    float *partial;   // rows of 2 D floats: dw's, then db's
    int64_t lddy, lds, ldds, lddx, rows;
    int D;
};

template <class T, int W, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) layer_grad_kernel(const LayerGradArgs a) {
    __shared__ float2 red[2][32];
    pdl_trigger();
    pdl_wait();
    const int64_t group = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t groups = (int64_t)gridDim.x * blockDim.y;
    Raw<T, W> vw[NV];
    float dw[NV][W], db[NV][W];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * W;
        vw[i] = load_or_zero<T, W>(static_cast<const T *>(a.w) + c, c < a.D);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[i][j] = db[i][j] = 0.f;
    }
    // every group of the CTA takes as many turns as its first one (barriers)
    const int64_t first = (int64_t)blockIdx.x * blockDim.y;
    const int turns = first < a.rows ? (int)((a.rows - 1 - first) / groups) + 1 : 0;
    // the next row's loads are issued before this row's sums where registers allow it
    constexpr bool AHEAD = MAXT <= 512;
    Raw<T, W> ny[NV], ns[NV];
    float nm = 0.f, nr = 0.f;
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
        }
        nm = live ? a.mean[row] : 0.f;
        nr = live ? a.rstd[row] : 0.f;
    };
    // where they do not, it is brought to L2 in the meantime, a lane a 128-byte line
    auto prefetch_row = [&](int64_t row) {
        constexpr int LANES = W * (int)sizeof(T) >= 4 ? 128 / (W * (int)sizeof(T)) : 32;
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
            if (AHEAD) vd[i] = load_ds(row, (i * blockDim.x + threadIdx.x) * W);
        }
        const float mean = nm, rstd = nr;
        if (AHEAD && t + 1 < turns) load_row(row + groups);
        float sg = 0.f, sgn = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float dy[W], s[W], w[W];
            vy[i].get(dy);
            vs[i].get(s);
            vw[i].get(w);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float n = (s[j] - mean) * rstd, g = dy[j] * w[j];
                sg += g;
                sgn = fmaf(g, n, sgn);
                dw[i][j] = fmaf(dy[j], n, dw[i][j]);
                db[i][j] += dy[j];
            }
        }
        // two buffers: a warp may reach the next turn's while another still reads this
        // one's, not the one after (that takes the next barrier)
        const float2 k = group_sum2(sg, sgn, red[t & 1]);
        const float kg = k.x / (float)a.D, kn = k.y / (float)a.D;
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
            for (int j = 0; j < W; ++j) {
                const float n = (s[j] - mean) * rstd;
                dx[j] = fmaf(rstd, fmaf(-n, kn, fmaf(dy[j], w[j], -kg)), ds[j]);
            }
            put<T, W>(static_cast<T *>(a.dX) + row * a.lddx + c, dx);
        }
    }
    if (a.partial == nullptr) return;
    // one row of partial sums a CTA: its groups' sums are added in their order (groups share a
    // CTA only up to 512 threads)
    __shared__ float sums[512 * NV * W];
    const int width = blockDim.x * NV * W;
    auto join = [&](float (&d)[NV][W]) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j)
                sums[threadIdx.y * width + (i * W + j) * blockDim.x + threadIdx.x] = d[i][j];
        __syncthreads();
        if (threadIdx.y == 0)
            for (int y = 1; y < (int)blockDim.y; ++y)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        d[i][j] += sums[y * width + (i * W + j) * blockDim.x + threadIdx.x];
        __syncthreads();
    };
    if (blockDim.y > 1) {
        join(dw);
        join(db);
        if (threadIdx.y > 0) return;
    }
    float *to = a.partial + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * W;
        if (c >= a.D) continue;   // (D is a multiple of W)
        if constexpr (W % 4 == 0) {
#pragma unroll
            for (int j = 0; j < W; j += 4) {
                *reinterpret_cast<float4 *>(to + c + j) =
                    make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
                *reinterpret_cast<float4 *>(to + a.D + c + j) =
                    make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                to[c + j] = dw[i][j];
                to[a.D + c + j] = db[i][j];
            }
        }
    }
}

// The same for rows off the boundary, two accesses a thread.  All of a group's rows are so by as
// much (a multiple of eight groups lies between two), so that a thread's columns stay; the groups
// of a CTA hold different ones, and their sums are added by columns.
template <class T>
__global__ void __launch_bounds__(512) layer_grad_shift_kernel(const LayerGradArgs a) {
    constexpr int W = 16 / sizeof(T), NV = 2;
    __shared__ float2 red[2][32];
    pdl_trigger();
    pdl_wait();
    const int64_t group = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t groups = (int64_t)gridDim.x * blockDim.y;
    const Shifted at = shifted<T, W>(static_cast<const T *>(a.S) + group * a.lds, a.D);
    const int end = at.end(W);
    const bool ends = end < a.D;
    auto access = [&](int i) { return i * (int)blockDim.x + (int)threadIdx.x; };
    auto column = [&](int i) { return access(i) * W + at.head; };
    auto in = [&](int i) { return access(i) < at.accesses; };
    Raw<T, W> vw[NV];
    float dw[NV][W], db[NV][W], end_dw = 0.f, end_db = 0.f;
    const float end_w = ends ? to_f32(static_cast<const T *>(a.w)[end]) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        vw[i] = load_moved<T, W>(static_cast<const T *>(a.w), access(i), at.head, in(i));
#pragma unroll
        for (int j = 0; j < W; ++j) dw[i][j] = db[i][j] = 0.f;
    }
    const int64_t first = (int64_t)blockIdx.x * blockDim.y;
    const int turns = first < a.rows ? (int)((a.rows - 1 - first) / groups) + 1 : 0;
    Raw<T, W> ny[NV], ns[NV];
    Raw<T, 1> end_ny, end_ns;
    float nm = 0.f, nr = 0.f;
    auto load_row = [&](int64_t row) {
        const bool live = row < a.rows;
        const T *dy = static_cast<const T *>(a.dY) + row * a.lddy;
        const T *s = static_cast<const T *>(a.S) + row * a.lds;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ny[i] = load_or_zero<T, W>(dy + column(i), live && in(i));
            ns[i] = load_or_zero<T, W>(s + column(i), live && in(i));
        }
        end_ny = load_or_zero<T, 1>(dy + end, live && ends);
        end_ns = load_or_zero<T, 1>(s + end, live && ends);
        nm = live ? a.mean[row] : 0.f;
        nr = live ? a.rstd[row] : 0.f;
    };
    if (turns > 0) load_row(group);
    for (int t = 0; t < turns; ++t) {
        const int64_t row = group + t * groups;
        const bool live = row < a.rows, stream = live && a.dS != nullptr;
        const T *more = static_cast<const T *>(a.dS) + row * a.ldds;
        Raw<T, W> vy[NV], vs[NV], vd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            vy[i] = ny[i];
            vs[i] = ns[i];
            vd[i] = load_or_zero<T, W>(more + column(i), stream && in(i));
        }
        const Raw<T, 1> end_d = load_or_zero<T, 1>(more + end, stream && ends);
        const float end_y = to_f32(end_ny.u), end_s = to_f32(end_ns.u);
        const float mean = nm, rstd = nr;
        if (t + 1 < turns) load_row(row + groups);
        float sg = 0.f, sgn = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float dy[W], s[W], w[W];
            vy[i].get(dy);
            vs[i].get(s);
            vw[i].get(w);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float n = (s[j] - mean) * rstd, g = dy[j] * w[j];
                sg += g;
                sgn = fmaf(g, n, sgn);
                dw[i][j] = fmaf(dy[j], n, dw[i][j]);
                db[i][j] += dy[j];
            }
        }
        const float end_n = (end_s - mean) * rstd, end_g = end_y * end_w;
        if (ends) {
            sg += end_g;
            sgn = fmaf(end_g, end_n, sgn);
            end_dw = fmaf(end_y, end_n, end_dw);
            end_db += end_y;
        }
        const float2 k = group_sum2(sg, sgn, red[t & 1]);   // (as above)
        const float kg = k.x / (float)a.D, kn = k.y / (float)a.D;
        if (!live) continue;
        T *to = static_cast<T *>(a.dX) + row * a.lddx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in(i)) continue;
            float dy[W], s[W], w[W], ds[W], dx[W];
            vy[i].get(dy);
            vs[i].get(s);
            vw[i].get(w);
            vd[i].get(ds);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float n = (s[j] - mean) * rstd;
                dx[j] = fmaf(rstd, fmaf(-n, kn, fmaf(dy[j], w[j], -kg)), ds[j]);
            }
            put<T, W>(to + column(i), dx);
        }
        if (ends)
            to[end] = from_f32<T>(fmaf(rstd, fmaf(-end_n, kn, end_g - kg), to_f32(end_d.u)));
    }
    if (a.partial == nullptr) return;
    __shared__ float sums[512 * NV * W + 16 * W];   // D a group, of up to 16 groups
    float *mine = sums + threadIdx.y * a.D;
    auto join = [&](const float (&d)[NV][W], float end_d, float *to) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (in(i)) mine[column(i) + j] = d[i][j];
        if (ends) mine[end] = end_d;
        __syncthreads();
        for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < a.D; c += blockDim.x * blockDim.y) {
            float sum = sums[c];
            for (int y = 1; y < (int)blockDim.y; ++y) sum += sums[y * a.D + c];
            to[c] = sum;
        }
        __syncthreads();
    };
    float *to = a.partial + (int64_t)blockIdx.x * 2 * a.D;
    join(dw, end_dw, to);
    join(db, end_db, to + a.D);
}

// The same where rows are long and many.  What bounded it there was the turn: about twenty
// instructions an element, in two phases that all of an SM's warps took together.  So here
//   - a group's rows come by bulk copies into a ring of its own in shared memory, up to three rows
//     ahead (issued by the group's first warp), and take no registers before they are used;
//   - groups meet in barriers of their own, so that one's sums run beside another's products;
//   - the arithmetic is in pairs (packed fp32), the weights stay in fp32.
// (16384 x 4096 bf16 with the stream's gradient: 95 us by the kernel above, 89 here.)
//   full[group, stage]: a row has landed; the group's barrier of a turn, which the sums need
//   anyway, also says that the row before it has been read to its end: its stage is filled again.
// Waits are bounded; one that runs out raises the library's status word, and the group goes on
// (without waiting again) to its end, as all barriers are met whatever was read.
struct LayerRingArgs {
    LayerGradArgs g;
    int tpr, groups, stages;
    unsigned *error;
};
constexpr int kRingThreads = 512;
constexpr int kRingBytes = 208 * 1024, kWideRingBytes = 225 * 1024;
constexpr int kRingStages = 4;

// An access's elements as pairs.
template <class T, int W>
__device__ __forceinline__ void pairs(const Raw<T, W> &r, float2 (&f)[W / 2]) {
    float v[W];
    r.get(v);
#pragma unroll
    for (int j = 0; j < W / 2; ++j) f[j] = make_float2(v[2 * j], v[2 * j + 1]);
}

// WIDE: 32 columns a thread, for which registers hold the columns' sums only: a row is read from the
// ring again for its products, the weights from L2 (16-bit rows beyond 8192 columns: 8192 x 12288 bf16
// 383 us in 1024 threads of 16 columns, whose 64 registers spill, 183 here).
template <class T, bool WIDE>
__global__ void __launch_bounds__(kRingThreads, 1) layer_grad_ring_kernel(const LayerRingArgs args) {
    constexpr int W = 16 / sizeof(T), NV = (WIDE ? 32 : 16) / W, P = W / 2;   // 16 columns a thread
    const LayerGradArgs &a = args.g;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float red[2][2][16];
    __shared__ uint64_t full[16 * kRingStages];
    __shared__ int abort_word;
    volatile int *abort = &abort_word;
    const int tpr = args.tpr, groups = args.groups, stages = args.stages;
    const int row_bytes = a.D * (int)sizeof(T), streams = a.dS != nullptr ? 3 : 2;
    if (threadIdx.x < 16 * kRingStages)
        tc::mbar_init(tc::smem_u32_generic(full + threadIdx.x), 1);
    if (threadIdx.x == 0) *abort = 0;
    tc::fence_barrier_init();
    pdl_trigger();
    __syncthreads();
    pdl_wait();
    const int y = threadIdx.x / tpr, x = threadIdx.x - y * tpr, warps = tpr >> 5;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool mine = y < groups;
    // this group's rows row0, row0 + step, ...
    const int64_t row0 = (int64_t)blockIdx.x * groups + y, step = (int64_t)gridDim.x * groups;
    const int turns = mine && row0 < a.rows ? (int)((a.rows - 1 - row0) / step) + 1 : 0;
    const uint32_t full0 = tc::smem_u32_generic(full + (mine ? y * kRingStages : 0));
    const T *const rows = reinterpret_cast<const T *>(ring + (mine ? y : 0) * stages * streams * row_bytes);
    auto issue = [&](int t) {   // by the group's first warp, a stream a lane
        const int s = t % stages;
        const int64_t row = row0 + t * step;
        if (lane == 0) tc::mbar_arrive_expect_tx(full0 + 8 * s, (uint32_t)(streams * row_bytes));
        __syncwarp();
        if (lane < streams) {
            const T *from = lane == 0   ? static_cast<const T *>(a.dY) + row * a.lddy
                            : lane == 1 ? static_cast<const T *>(a.S) + row * a.lds
                                        : static_cast<const T *>(a.dS) + row * a.ldds;
            const uint32_t to = tc::smem_u32_generic(rows) + (uint32_t)((s * streams + lane) * row_bytes);
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
                         " [%0], [%1], %2, [%3];"
                         :: "r"(to), "l"(from), "r"(row_bytes), "r"(full0 + 8 * s) : "memory");
        }
        __syncwarp();
    };
    if (x < 32)
        for (int t = 0; t < min(stages, turns); ++t) issue(t);
    float2 w[WIDE ? 1 : NV][P], dw[NV][P], db[NV][P];
    auto load_weights = [&](int c, float2 (&w)[P]) {
        pairs<T, W>(load_or_zero<T, W>(static_cast<const T *>(a.w) + c, mine && c < a.D), w);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + x) * W;
        if constexpr (!WIDE) load_weights(c, w[i]);
#pragma unroll
        for (int j = 0; j < P; ++j) dw[i][j] = db[i][j] = make_float2(0.f, 0.f);
    }
    float next_mean = 0.f, next_rstd = 0.f;
    auto load_statistics = [&](int t) {
        if (t >= turns) return;
        next_mean = a.mean[row0 + t * step];
        next_rstd = a.rstd[row0 + t * step];
    };
    load_statistics(0);
    for (int t = 0; t < turns; ++t) {
        const int64_t row = row0 + t * step;
        const float2 mean = make_float2(-next_mean, -next_mean), rstd = make_float2(next_rstd, next_rstd);
        load_statistics(t + 1);
        const T *dy = rows + (t % stages) * streams * a.D, *s = dy + a.D, *ds = s + a.D;
        (void)tc::wait(full0 + 8 * (t % stages), (t / stages) & 1, abort);
        Raw<T, W> vy[WIDE ? 1 : NV], vs[WIDE ? 1 : NV];
        float2 sg = make_float2(0.f, 0.f), sgn = sg;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + x) * W, held = WIDE ? 0 : i;
            if constexpr (WIDE) load_weights(c, w[0]);
            vy[held] = load_or_zero<T, W>(dy + c, c < a.D);
            vs[held] = load_or_zero<T, W>(s + c, c < a.D);
            float2 fy[P], fs[P];
            pairs<T, W>(vy[held], fy);
            pairs<T, W>(vs[held], fs);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 n = __fmul2_rn(__fadd2_rn(fs[j], mean), rstd);
                const float2 g = __fmul2_rn(fy[j], w[held][j]);
                sg = __fadd2_rn(sg, g);
                sgn = __ffma2_rn(g, n, sgn);
                dw[i][j] = __ffma2_rn(fy[j], n, dw[i][j]);
                db[i][j] = __fadd2_rn(db[i][j], fy[j]);
            }
        }
        // the lower half of the warp adds up g, the upper one g n
        const bool upper = lane >= 16;
        float k = (upper ? sgn.x + sgn.y : sg.x + sg.y) +
                  __shfl_xor_sync(0xffffffffu, upper ? sg.x + sg.y : sgn.x + sgn.y, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
        if (warps > 1) {
            // two buffers: a warp may reach the next turn's while another still reads this one's
            if ((lane & 15) == 0) red[t & 1][lane >> 4][warp] = k;
            asm volatile("bar.sync %0, %1;" :: "r"(1 + y), "r"(tpr) : "memory");
            k = (lane & 15) < warps ? red[t & 1][lane >> 4][y * warps + (lane & 15)] : 0.f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
        } else {
            __syncwarp();
        }
        // (the mean by a division: a rounded 1 / D would double its error)
        k = -rstd.x * (k / (float)a.D);
        const float kg = __shfl_sync(0xffffffffu, k, 0), kn = __shfl_sync(0xffffffffu, k, 16);
        if (x < 32 && t > 0 && t - 1 + stages < turns) issue(t - 1 + stages);
        // dx = ds - rstd mean g + rstd g - rstd mean(g n) n
        const float2 kg2 = make_float2(kg, kg), kn2 = make_float2(kn, kn);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + x) * W, held = WIDE ? 0 : i;
            if (c >= a.D) continue;
            float2 fy[P], fs[P], fd[P];
            float dx[W];
            if constexpr (WIDE) {
                load_weights(c, w[0]);
                vy[0].load(dy + c);
                vs[0].load(s + c);
            }
            pairs<T, W>(vy[held], fy);
            pairs<T, W>(vs[held], fs);
            pairs<T, W>(load_or_zero<T, W>(ds + c, streams == 3), fd);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 n = __fmul2_rn(__fadd2_rn(fs[j], mean), rstd);
                const float2 g = __fmul2_rn(fy[j], w[held][j]);
                const float2 d = __ffma2_rn(n, kn2, __ffma2_rn(g, rstd, kg2));
                dx[2 * j] = d.x + fd[j].x;
                dx[2 * j + 1] = d.y + fd[j].y;
            }
            put<T, W>(static_cast<T *>(a.dX) + row * a.lddx + c, dx);
        }
    }
    if (*abort && x < 32) {   // an aborted group does not leave with copies in flight
        int ignored = 0;
        for (int t = max(0, turns - stages); t < turns; ++t)
            (void)tc::mbar_wait(full0 + 8 * (t % stages), (t / stages) & 1, &ignored);
        if (x == 0 && args.error != nullptr) atomicOr(args.error, 1u);
    }
    __syncthreads();   // the ring is free
    if (a.partial == nullptr) return;
    // one row of partial sums a CTA: its groups' sums are added in their order
    float2 *sums = reinterpret_cast<float2 *>(ring);
    const int width = tpr * NV * P;
    auto join = [&](float2 (&d)[NV][P]) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (mine) sums[y * width + (i * P + j) * tpr + x] = d[i][j];
        __syncthreads();
        if (y == 0)
            for (int k = 1; k < groups; ++k)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        d[i][j] = __fadd2_rn(d[i][j], sums[k * width + (i * P + j) * tpr + x]);
        __syncthreads();
    };
    if (groups > 1) {
        join(dw);
        join(db);
    }
    if (y > 0) return;
    float *to = a.partial + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + x) * W;
        if (c >= a.D) continue;
#pragma unroll
        for (int j = 0; j < P; j += 2) {
            *reinterpret_cast<float4 *>(to + c + 2 * j) =
                make_float4(dw[i][j].x, dw[i][j].y, dw[i][j + 1].x, dw[i][j + 1].y);
            *reinterpret_cast<float4 *>(to + a.D + c + 2 * j) =
                make_float4(db[i][j].x, db[i][j].y, db[i][j + 1].x, db[i][j + 1].y);
        }
    }
}

// Rows wider than a group's registers: the CTA reads each of its rows twice and keeps its
// columns' sums in its own row of the workspace.
template <class T>
__global__ void __launch_bounds__(kMaxThreads) layer_grad_wide_kernel(const LayerGradArgs a) {
    __shared__ float2 red[2][32];
    pdl_trigger();
    pdl_wait();
    const T *w = static_cast<const T *>(a.w);
    float *part = a.partial != nullptr ? a.partial + (int64_t)blockIdx.x * 2 * a.D : nullptr;
    int t = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++t) {
        const T *dy = static_cast<const T *>(a.dY) + row * a.lddy;
        const T *s = static_cast<const T *>(a.S) + row * a.lds;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float sg = 0.f, sgn = 0.f;
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            const float g = to_f32(dy[c]) * to_f32(w[c]);
            sg += g;
            sgn = fmaf(g, (to_f32(s[c]) - mean) * rstd, sgn);
        }
        const float2 k = group_sum2(sg, sgn, red[t & 1]);
        const float kg = k.x / (float)a.D, kn = k.y / (float)a.D;
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            const float y = to_f32(dy[c]), n = (to_f32(s[c]) - mean) * rstd;
            float dx = rstd * fmaf(-n, kn, fmaf(y, to_f32(w[c]), -kg));
            if (a.dS != nullptr) dx += to_f32(static_cast<const T *>(a.dS)[row * a.ldds + c]);
            if (part != nullptr) {
                part[c] = fmaf(y, n, t > 0 ? part[c] : 0.f);
                part[a.D + c] = y + (t > 0 ? part[a.D + c] : 0.f);
            }
            static_cast<T *>(a.dX)[row * a.lddx + c] = from_f32<T>(dx);
        }
    }
}

// ------------------------------------------------------------------ host side

template <class T, int W, int NV, bool QUANT, bool SHIFT = false>
cudaError_t launch_row(const LayerRowArgs &a, Shape sh, cudaStream_t s) {
    const dim3 grid((unsigned)((a.rows + sh.groups - 1) / sh.groups));
    const dim3 block((unsigned)sh.tpr, (unsigned)sh.groups);
    if (sh.tpr <= 512 && !SHIFT)
        return launch(layer_row_kernel<T, W, NV, SHIFT ? kMaxThreads : 512, QUANT, SHIFT>, grid, block, a, s);
    return launch(layer_row_kernel<T, W, NV, kMaxThreads, QUANT, SHIFT>, grid, block, a, s);
}

// Widest access of a call's rows, in elements: 16 bytes down to one element, by halves.
template <class... M>
int access_of(int size, int64_t D, const M &...aligned) {
    for (int w = 16 / size; w > 1; w /= 2)
        if (D % w == 0 && (aligned(w) && ...)) return w;
    return 1;
}

// NV accesses of W elements a thread.  Rows of one element an access that need more than 512
// threads at eight take sixteen: one CTA an SM would wait for each of its phases alone.
template <class T, int W, bool QUANT>
cudaError_t row_accesses(const LayerRowArgs &a, cudaStream_t s) {
    constexpr bool WHOLE = W * sizeof(T) == 16;
    const int64_t n = a.D / W;
    // few rows: as many threads as possible on each, for its latency (1 x 1001 bf16 4.3 -> 3.1 us)
    Shape sh = shape_for(n, 1);
    if (sh.tpr > 0 && a.rows <= 304) return launch_row<T, W, 1, QUANT>(a, sh, s);
    constexpr int NV = WHOLE ? 4 : W * sizeof(T) == 8 ? 4 : 8;
    sh = shape_for(n, NV);
    if (sh.tpr > 0 && (WHOLE || sh.tpr <= 512)) return launch_row<T, W, NV, QUANT>(a, sh, s);
    if constexpr (!WHOLE) {
        sh = shape_for(n, 2 * NV);
        if (sh.tpr > 0) return launch_row<T, W, 2 * NV, QUANT>(a, sh, s);
    }
    return launch(layer_row_wide_kernel<T, QUANT>, dim3((unsigned)a.rows), dim3(kMaxThreads), a, s);
}

// Elements that p lies past a boundary of 16 bytes' worth of the rows' elements (8-bit outputs: of
// as many bytes).
int past(const void *p, int size, int whole) {
    return (int)(reinterpret_cast<uintptr_t>(p) / size % whole);
}

template <class T, bool QUANT>
cudaError_t row_dispatch(const LayerRowArgs &a, cudaStream_t s) {
    constexpr int size = sizeof(T);
    const int w = access_of(size, a.D, [&](int w) {
        return aligned_to(a.X, a.ldx, size, w) && aligned_to(a.R, a.ldr, size, w) &&
               aligned_to(a.w, 0, size, w) && aligned_to(a.b, 0, size, w) &&
               aligned_to(a.S, a.lds, size, w) && aligned_to(a.Y, a.ldy, QUANT ? 1 : size, w);
    });
    constexpr int W = 16 / size;
    if (w == W) return row_accesses<T, W, QUANT>(a, s);
    if (w == W / 2) return row_accesses<T, W / 2, QUANT>(a, s);
    // Rows that take narrower accesses yet lie alike: from a boundary of its own for each row
    // (1280 x 6427 bf16 40.6 -> 14.7 us, f32 49.5 -> 26.4; 6428 in 8-byte accesses 13.8, else
    // 17.7), but few and short ones by one narrow access a thread (16 x 777 3.0, else 3.4), and
    // rows of less than 1 KB, whose ends would weigh too much (20000 x 77 13.8, else 22.1).
    const bool narrow = (a.rows <= 304 && a.D / w <= kMaxThreads) || a.D * size < 1024;
    const int m = past(a.X, size, W);
    auto alike = [&](const void *p, int64_t ld, int size) {
        return p == nullptr || (past(p, size, W) == m && (ld - a.ldx) % W == 0);
    };
    if (!narrow && alike(a.R, a.ldr, size) && alike(a.S, a.lds, size) &&
        alike(a.Y, a.ldy, QUANT ? 1 : size) && aligned_to(a.w, 0, size, W) &&
        aligned_to(a.b, 0, size, W)) {
        Shape sh = shape_for(a.D / W, 1);
        if (sh.tpr > 0 && a.rows <= 304) return launch_row<T, W, 1, QUANT, true>(a, sh, s);
        sh = shape_for(a.D / W, 4);
        if (sh.tpr > 0) return launch_row<T, W, 4, QUANT, true>(a, sh, s);
    }
    if constexpr (size == 2)
        if (w == 2) return row_accesses<T, 2, QUANT>(a, s);
    return row_accesses<T, 1, QUANT>(a, s);
}

template <bool QUANT>
cudaError_t row_types(int type, const LayerRowArgs &a, cudaStream_t s) {
    if (type == SGEMM_F32) return row_dispatch<float, QUANT>(a, s);
    if (type == SGEMM_BF16) return row_dispatch<__nv_bfloat16, QUANT>(a, s);
    return row_dispatch<__half, QUANT>(a, s);
}

// The backward pass's row groups: as many CTAs as the SMs hold at once, at most one group
// a row.
struct GradShape {
    int w, nv;      // elements an access, accesses a thread; nv 0: the wide kernel
    Shape sh;
    int ctas;
    bool ring, wide, shift;   // wide: the ring's 32 columns a thread
};
// Whether the ring takes rows of 16-byte pieces: of 1 KB or more (shorter rows would be many
// small copies) up to 512 threads' 16 columns, and enough of them for twenty turns a CTA, as it
// starts and ends later (ring / the other kernel, us: 16384 x 4096 bf16 89.5 / 95.0, 8192 x 4096
// 50.5 / 51.8, 4096 x 4096 31.4 / 30.5, 16384 x 1024 30.0 / 28.1, 5200 x 8192 66.3 / 68.0; f32 8192 x
// 4096 88.9 / 93.3, 2600 x 8192 68.6 / 62.5).  Widths whose groups leave many of the 512 threads idle,
// or are one a CTA, lose time here that others do not: 8192 rows of 4096 / 5120 / 6144 / 7168 / 8192
// bf16 columns 51 / 83 / 84 / 92 / 95 us, where their bytes take 40 / 50 / 59 / 69 / 79.
bool ring_takes(int type, int64_t rows, int64_t D, Shape sh) {
    return sh.tpr > 0 && sh.tpr <= 512 && D * dtype_size(type) >= 1024 &&
           rows >= 152 * 20 * (512 / sh.tpr);
}
GradShape grad_shape(int type, int64_t rows, int64_t D, int w, bool shift) {
    GradShape g = {};
    const bool whole = w * dtype_size(type) == 16;
    g.shift = shift;
    if (whole && !shift) {
        g.sh = shape_for(D / w, 16 / w);
        if (ring_takes(type, rows, D, g.sh)) {
            g.sh.groups = 512 / g.sh.tpr;
            g.w = w;
            g.nv = 16 / w;
            g.ctas = 152;
            g.ring = true;
            return g;
        }
        if (w == 8 && g.sh.tpr > 512) {   // up to 16384 columns
            g.sh = {shape_for(D / w, 4).tpr, 1};
            g.w = w;
            g.nv = 4;
            g.ctas = rows < 152 ? (int)rows : 152;
            g.ring = g.wide = true;
            return g;
        }
    }
    g.w = w;
    const int64_t n = shift ? D / w : (D + w - 1) / w;   // (a row's ends are no accesses)
    g.nv = whole ? 2 : w * dtype_size(type) == 8 ? 4 : 8;
    g.sh = shape_for(n, g.nv);
    if (g.sh.tpr == 0) {
        g.nv = 0;
        g.sh = {kMaxThreads, 1};
    }
    // one CTA of 512 threads an SM has half the partial sums of two of 256; its groups wait
    // for one another, so only where each takes eight turns or more (as in norm.cu)
    if (g.sh.tpr <= 256 && rows >= 152 * 8 * (512 / g.sh.tpr)) g.sh.groups = 512 / g.sh.tpr;
    const int64_t need = (rows + g.sh.groups - 1) / g.sh.groups;
    const int threads = g.sh.tpr * g.sh.groups;
    const int per_sm = threads > 512 ? 1 : 512 / threads;
    const int64_t most = (int64_t)152 * per_sm;
    g.ctas = (int)(need < most ? need : most);
    return g;
}

template <class T, bool WIDE>
cudaError_t launch_ring(const LayerGradArgs &a, const GradShape &g, cudaStream_t s) {
    constexpr int RING = WIDE ? kWideRingBytes : kRingBytes;
    static PerContext<bool> configured;
    bool done = false;
    if (!configured.get(current_context_id(), done)) {
        const cudaError_t e = cudaFuncSetAttribute(
            layer_grad_ring_kernel<T, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, RING);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    const int stage = g.sh.groups * (a.dS != nullptr ? 3 : 2) * a.D * (int)sizeof(T);
    const int stages = RING / stage < kRingStages ? RING / stage : kRingStages;
    const LayerRingArgs args = {a, g.sh.tpr, g.sh.groups, stages, device_error_word()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)g.ctas);
    cfg.blockDim = dim3(kRingThreads);
    cfg.dynamicSmemBytes = RING;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, layer_grad_ring_kernel<T, WIDE>, args);
}

template <class T>
cudaError_t grad_dispatch(const LayerGradArgs &a, const GradShape &g, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    if constexpr (W == 8)
        if (g.wide) return launch_ring<T, true>(a, g, s);
    if (g.ring) return launch_ring<T, false>(a, g, s);
    const dim3 grid((unsigned)g.ctas), block((unsigned)g.sh.tpr, (unsigned)g.sh.groups);
    if (g.shift) return launch(layer_grad_shift_kernel<T>, grid, block, a, s);
    if (g.nv == 0) return launch(layer_grad_wide_kernel<T>, grid, block, a, s);
    auto run = [&](auto w, auto nv) {
        return g.sh.tpr <= 512
                   ? launch(layer_grad_kernel<T, w(), nv(), 512>, grid, block, a, s)
                   : launch(layer_grad_kernel<T, w(), nv(), kMaxThreads>, grid, block, a, s);
    };
    using std::integral_constant;
    if constexpr (W == 8) {   // (more threads than 512: the ring)
        if (g.w == W) return launch(layer_grad_kernel<T, W, 2, 512>, grid, block, a, s);
    } else {
        if (g.w == W) return run(integral_constant<int, W>(), integral_constant<int, 2>());
    }
    if (g.w == W / 2) return run(integral_constant<int, W / 2>(), integral_constant<int, 4>());
    if constexpr (W == 8)
        if (g.w == 2) return run(integral_constant<int, 2>(), integral_constant<int, 8>());
    return run(integral_constant<int, 1>(), integral_constant<int, 8>());
}

}  // namespace
}  // namespace norm

cudaError_t launch_add_layernorm(int type, int64_t rows, int64_t D, const void *X, int64_t ldx,
                                 const void *R, int64_t ldr, const void *w, const void *b,
                                 float eps, void *S, int64_t lds, void *Y, int64_t ldy,
                                 float *q_scale, float *mean, float *rstd, cudaStream_t s) {
    const norm::LayerRowArgs a = {X,   R,   w,   b,    S,       Y,    ldx,  ldr,
                                  lds, ldy, rows, q_scale, mean, rstd, eps, (int)D};
    return q_scale != nullptr ? norm::row_types<true>(type, a, s)
                              : norm::row_types<false>(type, a, s);
}

// Rows of partial sums, the most of any access's plan (the caller's pointers decide which
// one runs).
int layernorm_backward_parts(int type, int64_t rows, int64_t D) {
    int most = 0;
    for (int w = 16 / dtype_size(type); w >= 1; w /= 2) {
        const int ctas = norm::grad_shape(type, rows, D, w, false).ctas;
        most = ctas > most ? ctas : most;
    }
    const int shifted = norm::grad_shape(type, rows, D, 16 / dtype_size(type), true).ctas;
    return shifted > most ? shifted : most;
}

cudaError_t launch_add_layernorm_backward(int type, int64_t rows, int64_t D, const void *dY,
                                          int64_t lddy, const void *S, int64_t lds,
                                          const float *mean, const float *rstd, const void *w,
                                          const void *dS, int64_t ldds, void *dX, int64_t lddx,
                                          void *dw, void *db, float *partial, cudaStream_t s) {
    const int size = dtype_size(type);
    const int width = norm::access_of(size, D, [&](int n) {
        using norm::aligned_to;
        return aligned_to(dY, lddy, size, n) && aligned_to(S, lds, size, n) &&
               aligned_to(w, 0, size, n) && aligned_to(dS, ldds, size, n) &&
               aligned_to(dX, lddx, size, n);
    });
    const int whole = 16 / size;
    norm::GradShape g = norm::grad_shape(type, rows, D, width, false);
    auto alike = [&](const void *p, int64_t ld) {
        return p == nullptr || (norm::past(p, size, whole) == norm::past(S, size, whole) &&
                                (ld - lds) % whole == 0);
    };
    // As in row_dispatch, but where the sums by columns at the end do not weigh more (1280 x 6427
    // bf16 57.6 -> 24.2 us, 8192 x 4097 280 -> 69.9, f32 262 -> 90.7, but 1000 x 1001 bf16 8.4 -> 9.5).
    if (width < whole / 2 && rows * D >= (1 << 21) && D * size >= 1024 && alike(dY, lddy) &&
        alike(dS, ldds) && alike(dX, lddx) && norm::aligned_to(w, 0, size, whole)) {
        const norm::GradShape from_boundary = norm::grad_shape(type, rows, D, whole, true);
        if (from_boundary.nv > 0 && from_boundary.sh.tpr <= 512) g = from_boundary;
    }
    const bool sums = dw != nullptr || db != nullptr;
    const norm::LayerGradArgs a = {dY,   S,    w,    dS,   dX,   mean, rstd, sums ? partial : nullptr,
                                   lddy, lds, ldds, lddx, rows, (int)D};
    cudaError_t e = type == SGEMM_F32    ? norm::grad_dispatch<float>(a, g, s)
                    : type == SGEMM_BF16 ? norm::grad_dispatch<__nv_bfloat16>(a, g, s)
                                         : norm::grad_dispatch<__half>(a, g, s);
    if (e != cudaSuccess || !sums) return e;
    return launch_column_sum2(type, partial, g.ctas, D, dw, db, 0, s);
}

}  // namespace sgemm
