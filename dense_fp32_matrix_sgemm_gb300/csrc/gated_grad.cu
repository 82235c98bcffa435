// What the gated layer's gradients need around the products: from dH and the stored
// pre-activations,
//   dZg = dH Zu act'(Zg),   dZu = dH act(Zg),
// with both bias gradients' column sums in the same pass, and the sum of two outputs'
// partial rows.  HBM bounds both: three reads and two writes an element (f32: two times
// three planes of 2 bytes written), each in 16-byte accesses.
// In the 16-bit types both dZ leave rounded to the type, as the tensor cores multiply 16-bit
// operands: held in two terms each they would double the products, which are nine tenths of the
// time.  It adds one rounding (2^-8 in bf16) to each term of the gradients' sums: of 2048 x 2048 x
// 1024 bf16 they are off by 2.35e-3 of their 2-norm, 1.66e-3 (their own rounding) with dZ in fp32,
// 2.9e-3 to 3.4e-3 where every step of the formula is rounded to bf16.  The biases' sums are of
// the unrounded values.
#include <cstdint>

#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "layer_math.cuh"
#include "layers.h"

namespace sgemm {
namespace gated {

constexpr int kThreads = 256;   // 32 column lanes x 8 row lanes
constexpr int kRowLanes = 8;

struct DzArgs {
    const void *dH, *Zg, *Zu;
    void *dZg, *dZu;
    float *partial;
    int64_t lddh, ldzg, ldzu, lddz;
    int64_t plane;   // f32: three bf16 planes this many elements apart; 0: dZ itself
    int M, N, act, rows_per_part;
    int chain;
};

// CTA (x, y): columns [32 W x, ...) of rows [y rows_per_part, ...), as dz_kernel.
template <class T, int W>
__global__ void __launch_bounds__(kThreads, 3) gated_dz_kernel(const DzArgs a) {
    __shared__ float red[kRowLanes][32 * W];
    chain_begin(a.chain);
    const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = (int)(blockIdx.x * 32 + lane) * W;
    const int r0 = (int)blockIdx.y * a.rows_per_part;
    const int r1 = min(a.M, r0 + a.rows_per_part);
    float sum[2][W];
#pragma unroll
    for (int j = 0; j < W; ++j) sum[0][j] = sum[1][j] = 0.f;
    if (c < a.N) {
        const T *dh = static_cast<const T *>(a.dH) + c;
        const T *zg = static_cast<const T *>(a.Zg) + c;
        const T *zu = static_cast<const T *>(a.Zu) + c;
        auto store = [&](void *base, int row, const float (&x)[W]) {
            if constexpr (sizeof(T) == 4) {
                if (a.plane != 0) {
                    put_planes<W>(static_cast<__nv_bfloat16 *>(base) + row * a.lddz + c, a.plane, x);
                    return;
                }
            }
            put<T, W>(static_cast<T *>(base) + row * a.lddz + c, x);
        };
        constexpr int U = 2;   // rows in flight
        for (int r = r0 + ty; r < r1; r += U * kRowLanes) {
            Raw<T, W> vh[U], vg[U], vu[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = r + u * kRowLanes;
                if (row < r1) {
                    vh[u].load(dh + row * a.lddh);
                    vg[u].load(zg + row * a.ldzg);
                    vu[u].load(zu + row * a.ldzu);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = r + u * kRowLanes;
                if (row >= r1) continue;
                float h[W], g[W], f[W];
                vh[u].get(h);
                vg[u].get(g);
                vu[u].get(f);
                float slope[W];
                activate_both_all<T>(g, slope, a.act);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    f[j] *= h[j] * slope[j];
                    g[j] *= h[j];
                    sum[0][j] += f[j];
                    sum[1][j] += g[j];
                }
                if (a.dZg != nullptr) {
                    store(a.dZg, row, f);
                    store(a.dZu, row, g);
                }
            }
        }
    }
    if (a.partial == nullptr) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k > 0) __syncthreads();   // the gate's sums have been read
#pragma unroll
        for (int j = 0; j < W; ++j) red[ty][lane * W + j] = sum[k][j];
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * W; i += kThreads) {
            const int col = (int)blockIdx.x * 32 * W + i;
            if (col >= a.N) break;
            float v = 0.f;
#pragma unroll
            for (int r = 0; r < kRowLanes; ++r) v += red[r][i];
            a.partial[((int64_t)blockIdx.y * 2 + k) * a.N + col] = v;
        }
    }
}

// 32 columns a CTA, 32 row lanes, as column_sum_kernel; blockIdx.y: which output.
template <class T>
__global__ void __launch_bounds__(1024) column_sum2_kernel(const float *partial, int parts,
                                                           int64_t N, T *out, T *out2, int chain) {
    __shared__ float red[32][33];
    chain_begin(chain);
    const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    T *const to = blockIdx.y == 0 ? out : out2;
    if (to != nullptr) {
        const float *from = partial + blockIdx.y * N;
        float v = 0.f;
        if (c < N) {
            constexpr int U = 10;   // rows in flight; up to 320 parts in one go
            for (int p0 = ty; p0 < parts; p0 += 32 * U) {
                float x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int p = p0 + 32 * u;
                    x[u] = p < parts ? __ldcg(from + 2 * p * N + c) : 0.f;   // (see chain_begin)
                }
#pragma unroll
                for (int u = 0; u < U; ++u) v += x[u];
            }
        }
        red[ty][lane] = v;
        __syncthreads();
        if (ty == 0 && c < N) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < 32; ++r) s += red[r][lane];
            to[c] = from_f32<T>(s);
        }
    }
    chain_end(chain);
}

// Rows copied to rows with 16-byte boundaries, up to three matrices a launch.  A warp takes 512
// bytes of a row at a time, a lane 16 of them: loads of the largest word that the source's
// rows allow (a lane's share their sectors through L1), one store.  Bytes past a row's end go
// to the destination's gap as zeros.  From piece to piece a warp steps without a division.
struct RepackArgs {
    RepackJob job[3];
    int blocks[3];
};
template <class U>
__device__ __forceinline__ void repack_rows(const RepackJob &j, int64_t warp, int64_t warps) {
    constexpr int N = 16 / sizeof(U);
    const int lane = threadIdx.x & 31;
    const int pieces = (int)((j.row_bytes + 511) / 512);
    const int64_t dr = warps / pieces;
    const int dc = (int)(warps - dr * pieces);
    int64_t r = warp / pieces;
    int pc = (int)(warp - r * pieces);
    for (; r < j.rows; r += dr, pc += dc) {
        if (pc >= pieces) {
            pc -= pieces;
            if (++r >= j.rows) break;
        }
        const int64_t at = (int64_t)pc * 512 + lane * 16;
        if (at >= j.row_bytes) continue;
        const char *from = static_cast<const char *>(j.src) + r * j.src_ld + at;
        U w[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[i] = at + i * (int)sizeof(U) < j.row_bytes
                       ? *reinterpret_cast<const U *>(from + i * sizeof(U)) : U{};
        uint4 v;
        if constexpr (sizeof(U) == 8) {
            v = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
        } else {
            uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < N; ++i)
                d[i * sizeof(U) / 4] |= (uint32_t)w[i] << (8 * (i * sizeof(U) % 4));
            v = make_uint4(d[0], d[1], d[2], d[3]);
        }
        *reinterpret_cast<uint4 *>(static_cast<char *>(j.dst) + r * j.dst_ld + at) = v;
    }
}
__global__ void __launch_bounds__(kThreads) repack3_kernel(const RepackArgs a) {
    pdl_trigger();
    pdl_wait();
    int block = (int)blockIdx.x, which = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (which == i && block >= a.blocks[i]) {
            block -= a.blocks[i];
            which = i + 1;
        }
    const RepackJob j = which == 0 ? a.job[0] : which == 1 ? a.job[1] : a.job[2];
    const int blocks = which == 0 ? a.blocks[0] : which == 1 ? a.blocks[1] : a.blocks[2];
    const int64_t warp = (int64_t)block * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t warps = (int64_t)blocks * (kThreads / 32);
    switch (j.word) {
        case 8: repack_rows<uint2>(j, warp, warps); break;
        case 4: repack_rows<uint32_t>(j, warp, warps); break;
        case 2: repack_rows<uint16_t>(j, warp, warps); break;
        default: repack_rows<uint8_t>(j, warp, warps); break;
    }
}

bool aligned_to(const void *p, int64_t ld, int size, int elements) {
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)(size * elements) == 0 && ld % elements == 0;
}

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int block, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <class T>
cudaError_t dz_types(const DzArgs &a, int w, int parts, cudaStream_t s) {
    const int strip = 32 * w;
    const dim3 grid((unsigned)((a.N + strip - 1) / strip), (unsigned)parts);
    if constexpr (sizeof(T) == 2) {
        if (w == 8) return launch(gated_dz_kernel<T, 8>, grid, kThreads, s, a);
        if (w == 2) return launch(gated_dz_kernel<T, 2>, grid, kThreads, s, a);
    }
    return w == 4 ? launch(gated_dz_kernel<T, 4>, grid, kThreads, s, a)
                  : launch(gated_dz_kernel<T, 1>, grid, kThreads, s, a);
}

}  // namespace gated

// Row chunks of the pass: three CTAs an SM over the column strips of 16-byte accesses, so
// that the last round of CTAs is as full as it can be, each chunk at least 32 rows (4 a
// warp).  (4096 x 8192 bf16 in 608 CTAs, as for four an SM, 81 us.)
int gated_parts(int type, int64_t M, int64_t N) {
    const int64_t strip = 512 / dtype_size(type), strips = (N + strip - 1) / strip, room = 152 * 3;
    const int64_t most = (M + 31) / 32 < 1024 ? (M + 31) / 32 : 1024;
    int64_t best = 1;
    auto rounds = [&](int64_t p) { return (strips * p + room - 1) / room; };
    for (int64_t p = 2; p <= most && strips * p <= 4 * room; ++p)
        if (rounds(p) * best < rounds(best) * p) best = p;
    return (int)best;
}

cudaError_t launch_gated_dz(int type, const void *dH, int64_t lddh, const void *Zg, int64_t ldzg,
                            const void *Zu, int64_t ldzu, int act, int M, int N, void *dZg,
                            void *dZu, int64_t lddz, int64_t plane, float *partial, int chain,
                            cudaStream_t s) {
    // the widest access that all rows allow: 16 bytes, for the 16-bit types 8 or 4, or one element
    // (what is written lies in the workspace, whose rows are aligned)
    using gated::aligned_to;
    const int size = dtype_size(type);
    auto all = [&](int w) {
        return N % w == 0 && aligned_to(dH, lddh, size, w) && aligned_to(Zg, ldzg, size, w) &&
               aligned_to(Zu, ldzu, size, w);
    };
    int w = 16 / size;
    while (w > 1 && !all(w)) w = size == 4 ? 1 : w / 2;
    const int parts = gated_parts(type, M, N);
    const gated::DzArgs a = {dH,   Zg,   Zu,    dZg, dZu, partial, lddh,
                             ldzg, ldzu, lddz, plane, M,  N,   act,     (M + parts - 1) / parts,
                             chain};
    if (type == SGEMM_F32) return gated::dz_types<float>(a, w, parts, s);
    if (type == SGEMM_BF16) return gated::dz_types<__nv_bfloat16>(a, w, parts, s);
    return gated::dz_types<__half>(a, w, parts, s);
}

// One launch for up to three matrices; the words are chosen here.
cudaError_t launch_repack3(const RepackJob *jobs, int count, cudaStream_t s) {
    gated::RepackArgs a = {};
    int blocks = 0;
    for (int i = 0; i < count; ++i) {
        RepackJob &j = a.job[i];
        j = jobs[i];
        const uintptr_t bits = reinterpret_cast<uintptr_t>(j.src) | (uintptr_t)j.src_ld |
                               (uintptr_t)j.row_bytes;
        j.word = bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
        const int64_t need = (j.rows * ((j.row_bytes + 511) / 512) + 7) / 8;
        a.blocks[i] = (int)(need < 152 * 8 ? need : 152 * 8);
        blocks += a.blocks[i];
    }
    return gated::launch(gated::repack3_kernel, dim3((unsigned)blocks), gated::kThreads, s, a);
}

cudaError_t launch_column_sum2(int type, const float *partial, int parts, int64_t N, void *out,
                               void *out2, int chain, cudaStream_t s) {
    const dim3 grid((unsigned)((N + 31) / 32), 2);
    if (type == SGEMM_F32)
        return gated::launch(gated::column_sum2_kernel<float>, grid, 1024, s, partial, parts, N,
                             static_cast<float *>(out), static_cast<float *>(out2), chain);
    if (type == SGEMM_BF16)
        return gated::launch(gated::column_sum2_kernel<__nv_bfloat16>, grid, 1024, s, partial,
                             parts, N, static_cast<__nv_bfloat16 *>(out),
                             static_cast<__nv_bfloat16 *>(out2), chain);
    return gated::launch(gated::column_sum2_kernel<__half>, grid, 1024, s, partial, parts, N,
                         static_cast<__half *>(out), static_cast<__half *>(out2), chain);
}

}  // namespace sgemm
