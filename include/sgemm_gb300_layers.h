/*
 * sgemm_gb300_layers.h -- the operators around a transformer block's matrix
 * products on NVIDIA GB300 (sm_103a): the linear layer with bias, activation
 * and residual in its epilogue, its gradients, the root-mean-square norm with
 * the residual's addition (output in the input's type or in 8 bits with a
 * scale a row), its gradients, and the row quantiser.
 *
 * Layout, ownership, streams and errors are as in sgemm_gb300.h: row-major
 * matrices with leading dimensions in elements, device pointers owned by the
 * caller, work enqueued on `stream` without synchronising, arguments checked
 * on the host before anything is enqueued (a violation returns a nonzero
 * sgemm_status, enqueues nothing, and sgemm_last_error() describes it), no
 * device memory allocated per call.  Pointers are aligned to their element
 * type.  Results are deterministic.  Sums, norms and statistics are held in
 * 32 bits; an output is rounded once (to nearest even).
 */
#ifndef SGEMM_GB300_LAYERS_H
#define SGEMM_GB300_LAYERS_H

#include <stdint.h>

#include "sgemm_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif
#if defined(__GNUC__)
#pragma GCC visibility push(default)
#endif

typedef enum {
    SGEMM_F32 = 0,
    SGEMM_BF16 = 1,
    SGEMM_F16 = 2,
    SGEMM_E4M3 = 3   /* 8-bit float, 4 exponent and 3 mantissa bits, no infinities, max 448 */
} sgemm_dtype;

typedef enum {
    SGEMM_ACT_NONE = 0,
    SGEMM_ACT_RELU = 1,       /* max(z, 0); its gradient at 0 is 0 */
    SGEMM_ACT_GELU = 2,       /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
    SGEMM_ACT_GELU_ERF = 3,   /* z (1 + erf(z / sqrt 2)) / 2 */
    SGEMM_ACT_SILU = 4        /* z / (1 + exp(-z)) */
} sgemm_activation;

/*
 * The linear layer:
 *   z[i,j] = x_scale[i] w_scale[j] sum_k X[i,k] opW[k,j] + bias[j]
 *   Y[i,j] = act(z[i,j]) + residual[i,j]
 * X is M x K (ldx >= K).  W is stored N x K when transW == 1 (one row per
 * output feature, ldw >= K) and K x N when transW == 0 (ldw >= N).
 *   dtype       type of X and W.
 *   x_scale     SGEMM_E4M3 only, required there: M floats, the value of one
 *   w_scale     unit of each row of X, and N floats, that of each output
 *               feature's row of W; NULL for the other types.
 *   bias        NULL or N values of out_dtype.
 *   residual    NULL or M x N values of out_dtype (ldr >= N); it may be Y
 *               itself (same ldr), not overlap it otherwise.
 *   out_dtype   type of Y, bias, residual and preact: dtype itself, or for
 *               SGEMM_E4M3 one of SGEMM_BF16, SGEMM_F16.
 *   preact      NULL, or M x N values (ldp >= N) that receive z rounded to
 *               out_dtype (for sgemm_linear_backward); it overlaps nothing.
 * SGEMM_E4M3 takes transW == 1 only.  f32 products are formed on the tensor
 * cores from operands written as three bf16 terms each (FP32 accuracy; elements
 * below 2^-110 are held to 2^-134, half a bf16's smallest step), or by FP32 FMAs
 * for up to 16 rows; 16- and 8-bit products are exact and summed in
 * fp32.  A NaN or infinity in X makes its own row's values non-finite, one in W
 * its own feature's; in f32 on the tensor cores an infinity gives NaN where the
 * formula's sum would be infinite (its terms are formed from the difference of
 * infinities).  Y and preact overlap neither X nor W.
 * M == 0 or N == 0 does nothing; K == 0 gives act(bias) + residual, whatever
 * the scales.
 *   workspace   caller-owned device memory of at least
 *               sgemm_linear_workspace_size(...) bytes for the same
 *               arguments, 256-byte aligned, not used by other work while
 *               this call runs; NULL when that is 0.
 */
int sgemm_linear(int dtype, int64_t M, int64_t N, int64_t K,
                 const void *X, int64_t ldx, const float *x_scale,
                 const void *W, int64_t ldw, int transW, const float *w_scale,
                 const void *bias, int activation, const void *residual, int64_t ldr,
                 int out_dtype, void *Y, int64_t ldy, void *preact, int64_t ldp,
                 void *workspace, uint64_t workspace_bytes, void *stream);

/* Workspace bytes of sgemm_linear.  Of X and W only the alignment is looked
 * at (rows that are not 16-byte aligned are copied into the workspace first,
 * with aligned rows).  0 when the call needs none. */
uint64_t sgemm_linear_workspace_size(int dtype, int64_t M, int64_t N, int64_t K,
                                     const void *X, int64_t ldx,
                                     const void *W, int64_t ldw, int transW);

/*
 * Gradients of the linear layer.  With dZ = dY * act'(Z):
 *   dX[i,k] = sum_j dZ[i,j] opW[k,j]     (M x K, lddx >= K)
 *   dW      = the gradient of W, stored as W is (transW, lddw)
 *   db[j]   = sum_i dZ[i,j]
 * (the residual's gradient is dY).  Each of dX, dW, db may be NULL: it is
 * then not computed.  Z (M x N, ldz >= N) is the stored pre-activation; it is
 * not read, and may be NULL, for SGEMM_ACT_NONE.  dtype is the type of every
 * matrix: SGEMM_F32, SGEMM_BF16 or SGEMM_F16.  For the 16-bit types dZ enters
 * the two products rounded to the type (db is summed from the unrounded
 * values).  Where z is infinite, act' is its limit, 0 or 1.  X is read for dW
 * only, W for dX only.  No output overlaps an
 * input or another output.
 */
int sgemm_linear_backward(int dtype, int64_t M, int64_t N, int64_t K,
                          const void *dY, int64_t lddy, const void *Z, int64_t ldz, int activation,
                          const void *X, int64_t ldx, const void *W, int64_t ldw, int transW,
                          void *dX, int64_t lddx, void *dW, int64_t lddw, void *db,
                          void *workspace, uint64_t workspace_bytes, void *stream);

/* Workspace bytes of sgemm_linear_backward with every gradient asked for. */
uint64_t sgemm_linear_backward_workspace_size(int dtype, int64_t M, int64_t N, int64_t K,
                                              const void *dY, int64_t lddy, int activation,
                                              const void *X, int64_t ldx,
                                              const void *W, int64_t ldw, int transW);

/*
 * Root-mean-square norm of every row, after the residual's addition:
 *   s = X + residual          (residual NULL: s = X)
 *   rstd = (mean_d s^2 + eps)^(-1/2)
 *   y = s * rstd * weight
 * All of rows x D; dtype (SGEMM_F32, SGEMM_BF16, SGEMM_F16) is the type of X,
 * residual, weight and S.  y is formed from the unrounded s.
 *   S        NULL, or rows x D values that receive s (lds >= D; it may be X
 *            or residual itself with the same leading dimension).
 *   q_scale  NULL: Y is rows x D of dtype.  Else `rows` floats, and Y is
 *            rows x D SGEMM_E4M3 codes: with a = max(max_d |y|, 1e-30),
 *            q_scale = a / 448 and Y = y (448 / a) rounded to nearest even,
 *            so that y is about Y * q_scale.
 *   rstd     NULL, or `rows` floats.
 * A NaN or infinity makes its own row's values as the formula gives them and
 * touches no other row.  Rows of no elements (D == 0) have the statistics of
 * a row of zeros: q_scale = 1e-30 / 448, rstd = eps^(-1/2).
 */
int sgemm_add_rmsnorm(int dtype, int64_t rows, int64_t D, const void *X, int64_t ldx,
                      const void *residual, int64_t ldr, const void *weight, float eps,
                      void *S, int64_t lds, void *Y, int64_t ldy, float *q_scale, float *rstd,
                      void *stream);

/*
 * Gradients of sgemm_add_rmsnorm, from the stored s and rstd:
 *   g = dY * weight
 *   dX = dS + rstd (g - s rstd^2 mean_d(g s))     the gradient of X and of the residual alike
 *   dweight[d] = sum_rows dY s rstd
 * dS (rows x D, ldds) is the gradient that reaches s on the residual stream;
 * NULL means zero.  dX may be dY or dS itself with the same leading
 * dimension.  dweight may be NULL.  The workspace holds partial sums of
 * dweight: sgemm_add_rmsnorm_backward_workspace_size bytes, 256-byte aligned.
 */
int sgemm_add_rmsnorm_backward(int dtype, int64_t rows, int64_t D, const void *dY, int64_t lddy,
                               const void *S, int64_t lds, const float *rstd, const void *weight,
                               const void *dS, int64_t ldds, void *dX, int64_t lddx,
                               void *dweight, void *workspace, uint64_t workspace_bytes,
                               void *stream);
uint64_t sgemm_add_rmsnorm_backward_workspace_size(int dtype, int64_t rows, int64_t D);

/*
 * Every row of X (rows x D of dtype SGEMM_F32, SGEMM_BF16 or SGEMM_F16) as
 * 8-bit codes with one scale: a = max(max_d |x|, 1e-30), scale = a / 448,
 * Q = x (448 / a) rounded to nearest even (SGEMM_E4M3, ldq >= D).  A NaN or
 * infinity reaches its row's a: that row's scale and codes are as the formula
 * gives them, no other row's change.
 * Rows of no elements (D == 0) have the scale of a row of zeros.
 */
int sgemm_quantize_rows(int dtype, int64_t rows, int64_t D, const void *X, int64_t ldx,
                        void *Q, int64_t ldq, float *scale, void *stream);

#if defined(__GNUC__)
#pragma GCC visibility pop
#endif
#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_LAYERS_H */
