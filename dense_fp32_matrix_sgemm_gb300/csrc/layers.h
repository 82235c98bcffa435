// Internal launch interface of the layer operators (include/sgemm_gb300_layers.h)
// between layers_api.cu, which validates, and the kernel translation units.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "sgemm_gb300_layers.h"

namespace sgemm {

__host__ __device__ inline int dtype_size(int t) {
    return t == SGEMM_F32 ? 4 : t == SGEMM_E4M3 ? 1 : 2;
}

// Whether a product of M rows runs on the CUDA cores (linear_rows.cu).  layers_api.cu.
bool on_cuda_cores(int type, int64_t M, int64_t N, int64_t K, int transW);

// Place of a launch among launches of a call that do not read one another's results:
// after, before such a launch (chain_begin in layer_math.cuh), and with half of the
// SMs for each of two products.
enum { kChainPrev = 1, kChainNext = 2, kChainHalf = 4 };

// What happens to an accumulator on its way to memory:
//   z = acc * (sx ? sx[row] * sw[col] : 1) + bias[col];  Z = z
//   Y = act(z) + R
// All of `type` elements except the scales.  vec: the most of 16 (16-bit types
// only), 4 and 1 elements that every base and leading dimension is aligned to.
struct LayerEpi {
    void *Y, *Z;
    const void *R, *bias;
    const float *sx, *sw;
    int64_t ldy, ldz, ldr;
    int M, N;
    int act;
    int type;
    int vec;
};

// What happens to the two accumulators of a gated layer:
//   z = acc * (sx ? sx[row] * s[col] : 1) + b[col] for the gate (g) and its factor (u)
//   H = act(zg) zu;  Zg = zg, Zu = zu where they are kept
// vec: 8 (16-bit types only: 16-byte accesses), 4, 2 (16-bit types) or 1 elements that every
// base and leading dimension is aligned to.
struct GatedEpi {
    void *H, *Zg, *Zu;
    const void *bg, *bu;
    const float *sx, *sg, *su;
    int64_t ldh, ldg, ldu;
    int M, N;
    int act;
    int type;
    int vec;
};

// One operand of the tensor-core product: P (reduction) x rows as stored.
// kmajor: element (row, k) at base[row*ld + k], else at base[k*ld + row].
struct TcOperand {
    const void *base;
    int64_t ld;
    bool kmajor;
};

// A product's sizes as launch_linear_tc and launch_linear_f32 take them.
struct ProductSize {
    int M, N, K;
};
// (gated_tc.cu, gated_f32.cu)  H = act(X Wg^T + bg) (X Wu^T + bu), operands as
// launch_linear_tc takes them; both weights stored in one order.
cudaError_t launch_gated_tc(int in_type, const TcOperand &X, const TcOperand &Wg,
                            const TcOperand &Wu, int K, const GatedEpi &epi, cudaStream_t s);
// D = A1 B1^T + A2 B2^T, each reduction K long (count 1: the first alone).  epi: Y alone.
cudaError_t launch_sum_tc(int in_type, const TcOperand (&A)[2], const TcOperand (&B)[2], int count,
                          int K, const LayerEpi &epi, int chain, cudaStream_t s);
// The gated product of few rows on the CUDA cores, one pass over both weights for each few of them
// (f32: 8 rows, the others 4): any type and alignment of weights stored by output features
// (transW == 1), f32 alone of weights stored K x N (cudaErrorInvalidValue for the others, which
// the tensor cores take as they are).  linear_rows.cu.
cudaError_t launch_gated_rows(int in_type, const void *X, int64_t ldx, const void *Wg, int64_t ldwg,
                              const void *Wu, int64_t ldwu, int transW, int K, const GatedEpi &epi,
                              cudaStream_t s);

// Whether the gated layer's two weight gradients, each of this size, are better planned for
// half of the SMs each.
bool gated_side_by_side(int in_type, const ProductSize &product);

// Whether two products of a chain are better run side by side than in turn.
bool linear_tc_side_by_side(int in_type, const ProductSize &a, const ProductSize &b);
bool linear_f32_side_by_side(const ProductSize &a, const ProductSize &b);

// D[row, col] = sum_k A(row, k) B(col, k) with the epilogue, 16-bit operands
// of one type (SGEMM_BF16, SGEMM_F16) or SGEMM_E4M3 (K-major only), every
// operand's base and rows 16-byte aligned.  linear_tc.cu.
cudaError_t launch_linear_tc(int in_type, const TcOperand &A, const TcOperand &B, int K,
                             const LayerEpi &epi, int chain, cudaStream_t s);

// The same product of few rows on the CUDA cores, one pass over W; any type
// and alignment, transW == 1 for the types other than f32.  linear_rows.cu.
cudaError_t launch_linear_rows(int in_type, const void *X, int64_t ldx, const void *W, int64_t ldw,
                               int transW, int K, const LayerEpi &epi, cudaStream_t s);

// f32 on the tensor cores (linear_f32.cu): every operand as three bf16 planes
// that sum to it, in the orientation it is stored in.
struct F32Operand {   // rows x cols as stored, and where its planes go
    const float *X;
    int64_t ld, rows, cols;
    void *planes;
};
struct F32Planes {    // planes of a stored rows x cols matrix
    const void *planes;
    int64_t rows, cols;
    bool kmajor;      // cols is the reduction
};
inline int64_t f32_plane_ld(int64_t cols) { return (cols + 63) / 64 * 64; }   // of a plane's rows
size_t f32_planes_bytes(int64_t rows, int64_t cols);
cudaError_t launch_f32_split(const F32Operand *x, int count, int chain, cudaStream_t s);   // one to three
// D[row, col] = sum_k A(row, k) B(col, k) with the epilogue (float).
cudaError_t launch_linear_f32(const F32Planes &A, const F32Planes &B, int K, const LayerEpi &epi,
                              int chain, cudaStream_t s);
cudaError_t launch_gated_f32(const F32Planes &X, const F32Planes &Wg, const F32Planes &Wu, int K,
                             const GatedEpi &epi, cudaStream_t s);
cudaError_t launch_sum_f32(const F32Planes (&A)[2], const F32Planes (&B)[2], int K,
                           const LayerEpi &epi, int chain, cudaStream_t s);

// Rows of `bytes_per_row` bytes copied to rows `dst_ld` bytes apart (dst
// 16-byte aligned rows; the gap after each row is not written).
cudaError_t launch_repack(const void *src, int64_t src_ld_bytes, int64_t rows, int64_t row_bytes,
                          int elem, void *dst, int64_t dst_ld_bytes, cudaStream_t s);

// dZ = dY * act'(Z) (not written when dZ is null; f32 with plane > 0: as planes
// that many elements apart, rows lddz elements apart) and partial column sums of dZ,
// `parts` rows of N floats (not formed when partial is null).
int grad_parts(int64_t M, int64_t N);
cudaError_t launch_linear_dz(int type, const void *dY, int64_t lddy, const void *Z, int64_t ldz,
                             int act, int M, int N, void *dZ, int64_t lddz, int64_t plane,
                             float *partial, int chain, cudaStream_t s);

// out[c] = sum over `parts` rows of partial[part][c], added in a fixed order.
cudaError_t launch_column_sum(int type, const float *partial, int parts, int64_t N, void *out,
                              int chain, cudaStream_t s);

// The gated layer's dZg = dH Zu act'(Zg) and dZu = dH act(Zg) (f32 with plane > 0: as
// planes) with partial column sums of both, `parts` rows of 2 N floats.  gated_grad.cu
int gated_parts(int type, int64_t M, int64_t N);
cudaError_t launch_gated_dz(int type, const void *dH, int64_t lddh, const void *Zg, int64_t ldzg,
                            const void *Zu, int64_t ldzu, int act, int M, int N, void *dZg,
                            void *dZu, int64_t lddz, int64_t plane, float *partial, int chain,
                            cudaStream_t s);
// Rows of row_bytes bytes copied to rows dst_ld bytes apart, both 16-byte aligned there.
struct RepackJob {
    const void *src;
    void *dst;
    int64_t src_ld, dst_ld, rows, row_bytes;   // bytes
    int word;                                  // set by the launch
};
cudaError_t launch_repack3(const RepackJob *jobs, int count, cudaStream_t s);   // one to three
// out[c] and out2[c] = sums over `parts` rows of partial[part][c] and partial[part][N + c],
// added in a fixed order; either output may be null.
cudaError_t launch_column_sum2(int type, const float *partial, int parts, int64_t N, void *out,
                               void *out2, int chain, cudaStream_t s);

// norm.cu
cudaError_t launch_add_rmsnorm(int type, int64_t rows, int64_t D, const void *X, int64_t ldx,
                               const void *R, int64_t ldr, const void *w, float eps, void *S,
                               int64_t lds, void *Y, int64_t ldy, float *q_scale, float *rstd,
                               cudaStream_t s);
cudaError_t launch_quantize_rows(int type, int64_t rows, int64_t D, const void *X, int64_t ldx,
                                 void *Q, int64_t ldq, float *scale, cudaStream_t s);
int rmsnorm_backward_parts(int type, int64_t rows, int64_t D);
cudaError_t launch_add_rmsnorm_backward(int type, int64_t rows, int64_t D, const void *dY,
                                        int64_t lddy, const void *S, int64_t lds,
                                        const float *rstd, const void *w, const void *dS,
                                        int64_t ldds, void *dX, int64_t lddx, void *dw,
                                        float *partial, cudaStream_t s);

// layernorm.cu
cudaError_t launch_add_layernorm(int type, int64_t rows, int64_t D, const void *X, int64_t ldx,
                                 const void *R, int64_t ldr, const void *w, const void *b,
                                 float eps, void *S, int64_t lds, void *Y, int64_t ldy,
                                 float *q_scale, float *mean, float *rstd, cudaStream_t s);
int layernorm_backward_parts(int type, int64_t rows, int64_t D);
cudaError_t launch_add_layernorm_backward(int type, int64_t rows, int64_t D, const void *dY,
                                          int64_t lddy, const void *S, int64_t lds,
                                          const float *mean, const float *rstd, const void *w,
                                          const void *dS, int64_t ldds, void *dX, int64_t lddx,
                                          void *dw, void *db, float *partial, cudaStream_t s);

// grad_clip.cu: Y null: the norm alone
size_t grad_clip_bytes(int64_t count, const int *types, const int64_t *sizes);
cudaError_t launch_grad_clip(int64_t count, const int *types, const int64_t *sizes,
                             const void *const *X, void *const *Y, float max_norm, float eps,
                             float *norm, double *partial, cudaStream_t s);

}  // namespace sgemm
