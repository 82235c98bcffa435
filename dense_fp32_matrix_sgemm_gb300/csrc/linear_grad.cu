// What the linear layer's gradients need around the two products: dZ = dY *
// act'(Z) with the bias gradient's column sums in the same pass, the sum of
// partial rows, and the copy that gives a tensor-core operand aligned rows.
// All three are bound by HBM: 16-byte accesses, each byte moved once.
#include <cstdint>

#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "layer_math.cuh"
#include "layers.h"

namespace sgemm {
namespace grad {

constexpr int kThreads = 256;   // 32 column lanes x 8 row lanes
constexpr int kRowLanes = 8;

struct DzArgs {
    const void *dY, *Z;
    void *dZ;
    float *partial;
    int64_t lddy, ldz, lddz;
    int64_t plane;   // f32: dZ is three bf16 planes this many elements apart; 0: dZ itself
    int M, N, act, rows_per_part;
    int chain;
};

// CTA (x, y): columns [32 W x, ...) of rows [y rows_per_part, ...).  Lane l of
// a warp holds W consecutive columns, warp r the rows r, r + 8, ...; the
// columns' sums stay in registers over the rows, the eight warps' sums are
// added through shared memory in warp order.  f32 dZ that only the tensor-core
// products read is written as their planes (6 bytes an element instead of 4
// written, 4 read and 6 written).  Four CTAs an SM, which the grid counts on
// (without the bound 2 or 3 fit: 4096 x 8192 bf16, GELU, the column sums alone 37.3
// us, so 33.8, and 28.5 with the gradient's constants multiplied out; 30.8 with
// slopes that are right to the ends of z's range; with dZ written 35, 201 MB at
// 5.7 TB/s).
template <class T, int W>
__global__ void __launch_bounds__(kThreads, 4) dz_kernel(const DzArgs a) {
    __shared__ float red[kRowLanes][32 * W];
    chain_begin(a.chain);
    const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = (int)(blockIdx.x * 32 + lane) * W;
    const int r0 = (int)blockIdx.y * a.rows_per_part;
    const int r1 = min(a.M, r0 + a.rows_per_part);
    float sum[W];
#pragma unroll
    for (int j = 0; j < W; ++j) sum[j] = 0.f;
    if (c < a.N) {
        const T *dy = static_cast<const T *>(a.dY) + c;
        const T *z = static_cast<const T *>(a.Z) + c;
        T *dz = static_cast<T *>(a.dZ) + c;
        constexpr int U = W == 8 ? 3 : 4;   // rows in flight (W = 8: with four, 64 registers spill)
        for (int r = r0 + ty; r < r1; r += U * kRowLanes) {
            Raw<T, W> vy[U], vz[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = r + u * kRowLanes;
                if (row < r1) {
                    vy[u].load(dy + row * a.lddy);
                    if (a.act != SGEMM_ACT_NONE) vz[u].load(z + row * a.ldz);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = r + u * kRowLanes;
                if (row >= r1) continue;
                float g[W];
                vy[u].get(g);
                if (a.act != SGEMM_ACT_NONE) {
                    float f[W];
                    vz[u].get(f);
#pragma unroll
                    for (int j = 0; j < W; ++j) g[j] *= activate_grad<T>(f[j], a.act);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) sum[j] += g[j];
                if constexpr (sizeof(T) == 4) {
                    if (a.plane != 0) {
                        put_planes<W>(static_cast<__nv_bfloat16 *>(a.dZ) + row * a.lddz + c, a.plane,
                                      g);
                        continue;
                    }
                }
                if (a.dZ != nullptr) put<T, W>(dz + row * a.lddz, g);
            }
        }
    }
    if (a.partial == nullptr) return;
#pragma unroll
    for (int j = 0; j < W; ++j) red[ty][lane * W + j] = sum[j];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * W; i += kThreads) {
        const int col = (int)blockIdx.x * 32 * W + i;
        if (col >= a.N) break;
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < kRowLanes; ++r) v += red[r][i];
        a.partial[(int64_t)blockIdx.y * a.N + col] = v;
    }
}

// 32 columns a CTA, 32 row lanes: lane group y adds rows y, y + 32, ... of the
// partial sums, then the 32 sums are added in order.
template <class T>
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *partial, int parts,
                                                          int64_t N, T *out, int chain) {
    __shared__ float red[32][33];
    chain_begin(chain);
    const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < N) {
        constexpr int U = 10;   // rows in flight; up to 320 parts in one go
        for (int p0 = ty; p0 < parts; p0 += 32 * U) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int p = p0 + 32 * u;
                x[u] = p < parts ? __ldcg(partial + p * N + c) : 0.f;   // (see chain_begin)
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
        out[c] = from_f32<T>(s);
    }
    chain_end(chain);
}

// Row copy in words of U bytes (the largest that source and rows allow).
template <class U>
__global__ void __launch_bounds__(256) repack_kernel(const char *src, int64_t src_ld, int64_t rows,
                                                     int64_t words, char *dst, int64_t dst_ld) {
    pdl_trigger();
    pdl_wait();
    const int64_t total = rows * words;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / words, w = i - r * words;
        *reinterpret_cast<U *>(dst + r * dst_ld + w * sizeof(U)) =
            *reinterpret_cast<const U *>(src + r * src_ld + w * sizeof(U));
    }
}

bool aligned16(const void *p, int64_t ld, int size) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0);
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
cudaError_t dz_types(const DzArgs &a, bool vec, int parts, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    const int strip = 32 * (vec ? W : 1);
    const dim3 grid((unsigned)((a.N + strip - 1) / strip), (unsigned)parts);
    return vec ? launch(dz_kernel<T, W>, grid, kThreads, s, a)
               : launch(dz_kernel<T, 1>, grid, kThreads, s, a);
}

}  // namespace grad

// Row chunks of the dZ pass: about four CTAs an SM over the column strips of
// 256, each chunk at least 32 rows (4 a warp).
int grad_parts(int64_t M, int64_t N) {
    const int64_t strips = (N + 255) / 256;
    int64_t parts = (152 * 4 + strips - 1) / strips;
    const int64_t most = (M + 31) / 32;
    if (parts > most) parts = most;
    if (parts > 1024) parts = 1024;
    return parts < 1 ? 1 : (int)parts;
}

cudaError_t launch_linear_dz(int type, const void *dY, int64_t lddy, const void *Z, int64_t ldz,
                             int act, int M, int N, void *dZ, int64_t lddz, int64_t plane,
                             float *partial, int chain, cudaStream_t s) {
    const int size = dtype_size(type), w = 16 / size;
    const bool vec = N % w == 0 && grad::aligned16(dY, lddy, size) &&
                     (act == SGEMM_ACT_NONE || grad::aligned16(Z, ldz, size)) &&
                     (plane != 0 || grad::aligned16(dZ, lddz, size));
    const int parts = grad_parts(M, N);
    const grad::DzArgs a = {dY,   Z,     dZ, partial, lddy, ldz,
                            lddz, plane, M,  N,       act,  (M + parts - 1) / parts, chain};
    if (type == SGEMM_F32) return grad::dz_types<float>(a, vec, parts, s);
    if (type == SGEMM_BF16) return grad::dz_types<__nv_bfloat16>(a, vec, parts, s);
    return grad::dz_types<__half>(a, vec, parts, s);
}

cudaError_t launch_column_sum(int type, const float *partial, int parts, int64_t N, void *out,
                              int chain, cudaStream_t s) {
    const dim3 grid((unsigned)((N + 31) / 32));
    if (type == SGEMM_F32)
        return grad::launch(grad::column_sum_kernel<float>, grid, 1024, s, partial, parts, N,
                            static_cast<float *>(out), chain);
    if (type == SGEMM_BF16)
        return grad::launch(grad::column_sum_kernel<__nv_bfloat16>, grid, 1024, s, partial, parts,
                            N, static_cast<__nv_bfloat16 *>(out), chain);
    return grad::launch(grad::column_sum_kernel<__half>, grid, 1024, s, partial, parts, N,
                        static_cast<__half *>(out), chain);
}

cudaError_t launch_repack(const void *src, int64_t src_ld_bytes, int64_t rows, int64_t row_bytes,
                          int elem, void *dst, int64_t dst_ld_bytes, cudaStream_t s) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(src) | (uintptr_t)src_ld_bytes |
                           (uintptr_t)row_bytes;
    const int word = bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : elem;
    const int64_t words = row_bytes / word;
    const int64_t need = (rows * words + 255) / 256;
    const dim3 grid((unsigned)(need < 152 * 16 ? need : 152 * 16));
    const char *from = static_cast<const char *>(src);
    char *to = static_cast<char *>(dst);
    switch (word) {
        case 8:
            return grad::launch(grad::repack_kernel<uint2>, grid, 256, s, from, src_ld_bytes, rows,
                                words, to, dst_ld_bytes);
        case 4:
            return grad::launch(grad::repack_kernel<uint32_t>, grid, 256, s, from, src_ld_bytes,
                                rows, words, to, dst_ld_bytes);
        case 2:
            return grad::launch(grad::repack_kernel<uint16_t>, grid, 256, s, from, src_ld_bytes,
                                rows, words, to, dst_ld_bytes);
        default:
            return grad::launch(grad::repack_kernel<uint8_t>, grid, 256, s, from, src_ld_bytes,
                                rows, words, to, dst_ld_bytes);
    }
}

}  // namespace sgemm
