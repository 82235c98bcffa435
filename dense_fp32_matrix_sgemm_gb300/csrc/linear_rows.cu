// The linear layer of few rows (a decoding step's tokens) on the CUDA cores.
//
// z[i,j] = sum_k X[i,k] W[j,k] with M small: every weight is read once and
// used M times, so HBM bounds it (2 M flops a weight against 4, 2 or 1
// bytes), and what counts is that enough 16-byte loads are in flight on
// every SM from the start.  The tensor cores would be idle between loads all
// the same, and FP32 FMAs (packed in pairs) keep up for the few rows that the
// launcher sends here.
//
// Measured in a graph with weights out of L2, one row, K = 4096, 1024 to 32768
// features: bf16 3.1 us and the bytes at 6.5 TB/s (4096: 8.2 us, 4.1 TB/s; 8192: 13.7;
// 32768: 43.3, 6.2 TB/s), so a launch's start is what is left there; e4m3 2.5 us and
// the bytes at 5.3 TB/s (4096: 5.7; 32768: 27.8, 4.8 TB/s), where the codes'
// conversion costs instructions too.
// Weights stored N x K (dot form): a warp takes two or four output features and
// walks K, each lane with 16-byte pieces of their rows of W and of the MR rows of
// X (X stays in L1).  Where the features alone would not fill the SMs, K is
// split over the warps of a CTA and their sums are added through shared
// memory, in warp order.
// f32 weights stored K x N (column form): a lane takes 16 bytes of consecutive
// features and walks k; K is split over the warps of a CTA and over a cluster
// of CTAs, and the sums are added through shared and distributed shared
// memory in rank order.
// Rows or bases that are not 16-byte aligned take one element an access.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "layer_math.cuh"
#include "layers.h"

namespace sgemm {
namespace rows {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// W elements of T loaded as one access (16 bytes, or one element), and their
// values as pairs of floats.
template <class T, int W>
struct Piece {
    static constexpr int PAIRS = W / 2;
    uint4 u;
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float2 (&f)[PAIRS]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if constexpr (W == 4) {
            f[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
            f[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
        } else if constexpr (W == 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = unpack2<T>(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = from_e4m3x2((uint16_t)(w[i] & 0xffffu));
                f[2 * i + 1] = from_e4m3x2((uint16_t)(w[i] >> 16));
            }
        }
    }
};
template <class T>
struct Piece<T, 1> {
    static constexpr int PAIRS = 1;
    T u;
    __device__ __forceinline__ void load(const T *p) { u = *p; }
    __device__ __forceinline__ void get(float2 (&f)[1]) const {
        if constexpr (std::is_same<T, uint8_t>::value)
            f[0] = make_float2(from_e4m3x2(u).x, 0.f);
        else
            f[0] = make_float2(to_f32(u), 0.f);
    }
};

struct Args {
    const void *X, *W;
    int64_t ldx, ldw;
    int K;
    int split;   // dot form: warps of a CTA that share a feature pair's K
    LayerEpi epi;
};

// Dot form.  Warp w of the CTA: features j0 .. j0 + F - 1 of group w / split, K
// pieces w % split of split.  Accumulators hold the sums over even and odd
// positions of the pieces apart (one packed FMA for both).  F is 4 for 2 to 4
// rows of f32, where each piece of X is then read from L1 for four features
// (4096 x 4096 weights, 4 rows: 24.5 -> 16.3 us), else 2 (16-bit, 2 rows: 9.0
// us, with four 9.8; f32, 8 rows: 25, with four 35, whose 196 registers leave
// too few warps).
template <class T, int MR>
constexpr int kFeatures = sizeof(T) == 4 && (MR == 2 || MR == 4) ? 4 : 2;

template <class T, class O, int W, int MR>
__global__ void __launch_bounds__(kThreads) dot_kernel(const Args a) {
    constexpr int F = kFeatures<T, MR>;
    constexpr int U = F == 2 && MR <= 2 ? 4 : 2;   // pieces in flight a feature
    constexpr int P = Piece<T, W>::PAIRS;
    constexpr int SUMS = F * MR;
    static_assert(SUMS <= 32, "a sum a lane");
    __shared__ float red[kWarps][SUMS];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = warp % a.split;
    const int j0 = F * (int)(blockIdx.x * (kWarps / a.split) + warp / a.split);
    const T *w[F];
#pragma unroll
    for (int f = 0; f < F; ++f)
        w[f] = static_cast<const T *>(a.W) + (int64_t)min(j0 + f, a.epi.N - 1) * a.ldw;
    const int groups = (a.epi.M + MR - 1) / MR;
    for (int g = blockIdx.y; g < groups; g += gridDim.y) {
        const int m0 = g * MR;
        float2 acc[F][MR];
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int m = 0; m < MR; ++m) acc[f][m] = make_float2(0.f, 0.f);
        if (j0 < a.epi.N) {
            const T *x[MR];
#pragma unroll
            for (int m = 0; m < MR; ++m)
                x[m] = static_cast<const T *>(a.X) + min(m0 + m, a.epi.M - 1) * a.ldx;
            const int step = a.split * 32 * W;
            auto use = [&](const Piece<T, W> (&raw)[F], int k) {
                float2 fw[F][P];
#pragma unroll
                for (int f = 0; f < F; ++f) raw[f].get(fw[f]);
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    Piece<T, W> px;
                    px.load(x[m] + k);
                    float2 fx[P];
                    px.get(fx);
#pragma unroll
                    for (int f = 0; f < F; ++f)
#pragma unroll
                        for (int i = 0; i < P; ++i)
                            acc[f][m] = __ffma2_rn(fw[f][i], fx[i], acc[f][m]);
                }
            };
            int k = (sub * 32 + lane) * W;
            for (; k + (U - 1) * step < a.K; k += U * step) {
                Piece<T, W> raw[U][F];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int f = 0; f < F; ++f) raw[u][f].load(w[f] + k + u * step);
#pragma unroll
                for (int u = 0; u < U; ++u) use(raw[u], k + u * step);
            }
            for (; k < a.K; k += step) {
                Piece<T, W> raw[F];
#pragma unroll
                for (int f = 0; f < F; ++f) raw[f].load(w[f] + k);
                use(raw, k);
            }
        }
        // lane i < SUMS keeps the sum of feature i / MR and row i % MR
        float mine = 0.f;
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                float v = acc[f][m].x + acc[f][m].y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == f * MR + m) mine = v;
            }
        if (a.split > 1) {
            __syncthreads();   // the previous group's sums have been read
            if (lane < SUMS) red[warp][lane] = mine;
            __syncthreads();
            if (sub == 0 && lane < SUMS)
                for (int s = 1; s < a.split; ++s) mine += red[warp + s][lane];
        }
        const int row = m0 + lane % MR, col = j0 + lane / MR;
        if (sub == 0 && lane < SUMS && row < a.epi.M && col < a.epi.N)
            finish1<O>(a.epi, row, col, mine);
    }
}

// Column form: CTA (x, y) of a cluster along x of `cluster_size` CTAs: columns
// [strip * 32 W, ...), k = rank * kWarps + warp + kWarps * size * i.  f32 only: 16-bit weights in this
// orientation go to the tensor cores, which take it as it is (4096 x 4096, one
// row: 10.5 us there, 24 here).
template <int W, int MR>
__global__ void __launch_bounds__(kThreads) column_kernel(const Args a) {
    constexpr int COLS = 32 * W;
    __shared__ __align__(16) float red[kWarps][MR][COLS];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int strip = (int)(blockIdx.x / size);
    const int c = strip * COLS + lane * W;
    const int groups = (a.epi.M + MR - 1) / MR;
    for (int g = blockIdx.y; g < groups; g += gridDim.y) {
        const int m0 = g * MR;
        float acc[MR][W];
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int j = 0; j < W; ++j) acc[m][j] = 0.f;
        if (c < a.epi.N) {
            const float *w = static_cast<const float *>(a.W) + c;
            const float *x[MR];
#pragma unroll
            for (int m = 0; m < MR; ++m)
                x[m] = static_cast<const float *>(a.X) + min(m0 + m, a.epi.M - 1) * a.ldx;
            const int step = kWarps * (int)size;
            constexpr int U = 4;
            for (int k = (int)rank * kWarps + warp; k < a.K; k += U * step) {
                Raw<float, W> vw[U];
                float vx[U][MR];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int ku = k + u * step;
                    if (ku < a.K) vw[u].load(w + (int64_t)ku * a.ldw);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int m = 0; m < MR; ++m) vx[u][m] = x[m][min(k + u * step, a.K - 1)];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (k + u * step >= a.K) break;
                    float f[W];
                    vw[u].get(f);
#pragma unroll
                    for (int m = 0; m < MR; ++m)
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            acc[m][j] = fmaf(vx[u][m], f[j], acc[m][j]);
                }
            }
        }
        // this CTA's sums into red[0], in warp order
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int j = 0; j < W; ++j) red[warp][m][j * 32 + lane] = acc[m][j];
        __syncthreads();
        for (int i = threadIdx.x; i < MR * COLS; i += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) s += red[q][i / COLS][i % COLS];
            red[0][i / COLS][i % COLS] = s;
        }
        if (size > 1) cluster_sync();
        else __syncthreads();
        // each CTA of the cluster finishes a share of the strip (position p of a
        // strip is column p % 32 * W + p / 32)
        for (int i = (int)rank * kThreads + threadIdx.x; i < MR * COLS;
             i += (int)size * kThreads) {
            const int m = i / COLS, p = i % COLS, col = strip * COLS + p % 32 * W + p / 32;
            const float s = size > 1 ? cluster_sum_f32(smem_u32(&red[0][m][p]), size)
                                     : red[0][m][p];
            if (m0 + m < a.epi.M && col < a.epi.N) finish1<float>(a.epi, m0 + m, col, s);
        }
        // red is written again, or the CTA ends, only after every peer has read it
        if (size > 1) cluster_sync();
        else __syncthreads();
    }
}

template <class K>
cudaError_t launch(K kernel, dim3 grid, int threads, int cluster, const Args &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

constexpr int kSms = 152;

template <class T, class O, int W, int MR>
cudaError_t run(Args a, int transW, cudaStream_t s) {
    const int groups = (a.epi.M + MR - 1) / MR;
    const unsigned gy = (unsigned)(groups < 65535 ? groups : 65535);
    if (transW) {
        // warps a group of features: until about 24 warps an SM are busy, each
        // with at least one piece of K a lane
        constexpr int F = kFeatures<T, MR>;
        const int64_t sets = (a.epi.N + F - 1) / F;
        a.split = 1;
        while (a.split < kWarps && sets * gy * a.split < kSms * 24 &&
               (int64_t)a.K > (int64_t)a.split * 32 * W)
            a.split *= 2;
        const int64_t per_cta = kWarps / a.split;
        return launch(dot_kernel<T, O, W, MR>, dim3((unsigned)((sets + per_cta - 1) / per_cta), gy),
                      kThreads, 1, a, s);
    }
    if constexpr (std::is_same<T, float>::value) {
        const int64_t strips = (a.epi.N + 32 * W - 1) / (32 * W);
        int size = 1;
        while (size < 8 && strips * gy * size < kSms * 2 && a.K > size * kWarps * 4) size *= 2;
        return launch(column_kernel<W, MR>, dim3((unsigned)(strips * size), gy), kThreads, size, a,
                      s);
    }
    return cudaErrorInvalidValue;
}

template <class T, class O, int W>
cudaError_t by_rows(const Args &a, int transW, cudaStream_t s) {
    if (a.epi.M == 1) return run<T, O, W, 1>(a, transW, s);
    if (a.epi.M == 2) return run<T, O, W, 2>(a, transW, s);
    if (a.epi.M <= 4 || sizeof(T) < 4) return run<T, O, W, 4>(a, transW, s);
    if constexpr (sizeof(T) == 4) return run<T, O, W, 8>(a, transW, s);
    return cudaErrorInvalidValue;
}

template <class T, class O>
cudaError_t by_alignment(const Args &a, int transW, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    auto ok = [](const void *p, int64_t ld) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)sizeof(T) % 16 == 0;
    };
    const bool vec = transW ? ok(a.X, a.ldx) && ok(a.W, a.ldw) && a.K % W == 0
                            : ok(a.W, a.ldw) && a.epi.N % W == 0;
    return vec ? by_rows<T, O, W>(a, transW, s) : by_rows<T, O, 1>(a, transW, s);
}

}  // namespace rows

cudaError_t launch_linear_rows(int in_type, const void *X, int64_t ldx, const void *W, int64_t ldw,
                               int transW, int K, const LayerEpi &epi, cudaStream_t s) {
    const rows::Args a = {X, W, ldx, ldw, K, 1, epi};
    switch (in_type) {
        case SGEMM_F32: return rows::by_alignment<float, float>(a, transW, s);
        case SGEMM_BF16: return rows::by_alignment<__nv_bfloat16, __nv_bfloat16>(a, transW, s);
        case SGEMM_F16: return rows::by_alignment<__half, __half>(a, transW, s);
        default:
            return epi.type == SGEMM_BF16 ? rows::by_alignment<uint8_t, __nv_bfloat16>(a, transW, s)
                                          : rows::by_alignment<uint8_t, __half>(a, transW, s);
    }
}

}  // namespace sgemm
