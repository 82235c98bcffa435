/*
 * sgemm_gb300_block.h -- the gated feed-forward block on NVIDIA GB300
 * (sm_103a): the gated linear layer (two projections, the activation and
 * their product in one kernel) and its gradients, the layer norm with the
 * residual's addition and its gradients, and the clipping of a list of
 * gradients by their common norm.
 *
 * Types, activations, layout, ownership, streams, errors and determinism are
 * as in sgemm_gb300_layers.h.
 */
#ifndef SGEMM_GB300_BLOCK_H
#define SGEMM_GB300_BLOCK_H

#include <stdint.h>

#include "sgemm_gb300_layers.h"

#ifdef __cplusplus
extern "C" {
#endif
#if defined(__GNUC__)
#pragma GCC visibility push(default)
#endif

/*
 * The gated linear layer:
 *   zg[i,j] = x_scale[i] gate_scale[j] sum_k X[i,k] opWg[k,j] + bias_gate[j]
 *   zu[i,j] = x_scale[i] up_scale[j]   sum_k X[i,k] opWu[k,j] + bias_up[j]
 *   H[i,j]  = act(zg[i,j]) zu[i,j]
 * X is M x K (ldx >= K).  Both weights are stored N x K when transW == 1 (one
 * row per output feature, ldwg, ldwu >= K) or both K x N when transW == 0
 * (ldwg, ldwu >= N); they may be halves of one matrix.
 *   dtype       type of X, Wg and Wu: SGEMM_F32, SGEMM_BF16, SGEMM_F16, or
 *               SGEMM_E4M3 (transW == 1 only).
 *   x_scale, gate_scale, up_scale   SGEMM_E4M3 only, required there: M, N and
 *               N floats; NULL for the other types.
 *   bias_gate, bias_up   each NULL or N values of out_dtype.
 *   out_dtype   type of H, the biases and the pre-activations: dtype itself,
 *               or for SGEMM_E4M3 one of SGEMM_BF16, SGEMM_F16.
 *   preact_gate, preact_up   each NULL, or M x N values that receive zg and zu
 *               rounded to out_dtype (for sgemm_gated_linear_backward).  H is
 *               formed from the unrounded ones.
 * H and the pre-activations overlap no input and not one another.  Accuracy,
 * NaN and infinities as in sgemm_linear, of each projection.
 * N is at most 2^29.  M == 0 or N == 0 does nothing; K == 0 gives
 * act(bias_gate) bias_up.
 *   workspace   sgemm_gated_linear_workspace_size(...) bytes for the same
 *               arguments, 256-byte aligned; NULL when that is 0.
 */
int sgemm_gated_linear(int dtype, int64_t M, int64_t N, int64_t K,
                       const void *X, int64_t ldx, const float *x_scale,
                       const void *Wg, int64_t ldwg, const float *gate_scale,
                       const void *Wu, int64_t ldwu, const float *up_scale, int transW,
                       const void *bias_gate, const void *bias_up, int activation,
                       int out_dtype, void *H, int64_t ldh,
                       void *preact_gate, int64_t ldpg, void *preact_up, int64_t ldpu,
                       void *workspace, uint64_t workspace_bytes, void *stream);

/* Workspace bytes of sgemm_gated_linear; of the matrices only the alignment is looked at. */
uint64_t sgemm_gated_linear_workspace_size(int dtype, int64_t M, int64_t N, int64_t K,
                                           const void *X, int64_t ldx, const void *Wg, int64_t ldwg,
                                           const void *Wu, int64_t ldwu, int transW);

/*
 * Gradients of the gated linear layer from dH and the stored pre-activations:
 *   dZg = dH Zu act'(Zg)       dZu = dH act(Zg)
 *   dX  = dZg opWg^T + dZu opWu^T     (M x K, lddx >= K; summed before it is rounded)
 *   dWg, dWu = the weights' gradients, stored as the weights are (transW)
 *   db_gate[j] = sum_i dZg[i,j]       db_up[j] = sum_i dZu[i,j]
 * Each of dX, dWg, dWu, db_gate, db_up may be NULL: it is then not computed.
 * dtype is the type of every matrix: SGEMM_F32, SGEMM_BF16 or SGEMM_F16.  For
 * the 16-bit types dZg and dZu enter the products rounded to the type (the
 * biases' sums are of the unrounded values).  Where zg is infinite (a stored one may
 * have left its type's range), act' and act are their limits: 0 and 0, or 1 and infinity.
 * X is read for dWg and dWu only, the weights for dX only.  No output overlaps an input
 * or another output.
 */
int sgemm_gated_linear_backward(int dtype, int64_t M, int64_t N, int64_t K,
                                const void *dH, int64_t lddh, const void *Zg, int64_t ldzg,
                                const void *Zu, int64_t ldzu, int activation,
                                const void *X, int64_t ldx, const void *Wg, int64_t ldwg,
                                const void *Wu, int64_t ldwu, int transW,
                                void *dX, int64_t lddx, void *dWg, int64_t lddwg,
                                void *dWu, int64_t lddwu, void *db_gate, void *db_up,
                                void *workspace, uint64_t workspace_bytes, void *stream);

/* Workspace bytes of sgemm_gated_linear_backward with every gradient asked for. */
uint64_t sgemm_gated_linear_backward_workspace_size(int dtype, int64_t M, int64_t N, int64_t K,
                                                    const void *X, int64_t ldx,
                                                    const void *Wg, int64_t ldwg,
                                                    const void *Wu, int64_t ldwu, int transW);

/*
 * Layer norm of every row, after the residual's addition:
 *   s = X + residual          (residual NULL: s = X)
 *   mean = mean_d s           rstd = (mean_d (s - mean)^2 + eps)^(-1/2)
 *   y = (s - mean) rstd weight + bias       (bias NULL: none)
 * All of rows x D; dtype (SGEMM_F32, SGEMM_BF16, SGEMM_F16) is the type of X,
 * residual, weight, bias and S.  y is formed from the unrounded s.
 *   S, q_scale, Y   as in sgemm_add_rmsnorm (8-bit codes when q_scale is given).
 *   mean, rstd      each NULL, or `rows` floats.
 * A NaN or infinity makes its own row's values as the formula gives them and
 * touches no other row.  A row's sums are formed in 32 bits: where sum_d (s - mean)^2 passes
 * 3.4e38 it is infinite and rstd 0.  Rows of no elements (D == 0) have mean 0, rstd =
 * eps^(-1/2) and the scale of a row of zeros.
 */
int sgemm_add_layernorm(int dtype, int64_t rows, int64_t D, const void *X, int64_t ldx,
                        const void *residual, int64_t ldr, const void *weight, const void *bias,
                        float eps, void *S, int64_t lds, void *Y, int64_t ldy, float *q_scale,
                        float *mean, float *rstd, void *stream);

/*
 * Gradients of sgemm_add_layernorm, from the stored s, mean and rstd:
 *   n = (s - mean) rstd       g = dY * weight
 *   dX = dS + rstd (g - mean_d g - n mean_d(g n))     the gradient of X and of the residual alike
 *   dweight[d] = sum_rows dY n         dbias[d] = sum_rows dY
 * dS (rows x D, ldds) is the gradient that reaches s on the residual stream;
 * NULL means zero.  dX may be dY or dS itself with the same leading dimension.
 * dweight and dbias may each be NULL.  The workspace holds their partial sums:
 * sgemm_add_layernorm_backward_workspace_size bytes, 256-byte aligned.
 */
int sgemm_add_layernorm_backward(int dtype, int64_t rows, int64_t D, const void *dY, int64_t lddy,
                                 const void *S, int64_t lds, const float *mean, const float *rstd,
                                 const void *weight, const void *dS, int64_t ldds, void *dX,
                                 int64_t lddx, void *dweight, void *dbias, void *workspace,
                                 uint64_t workspace_bytes, void *stream);
uint64_t sgemm_add_layernorm_backward_workspace_size(int dtype, int64_t rows, int64_t D);

/*
 * The norm of all elements of `count` tensors, and the tensors scaled so that
 * it is at most max_norm:
 *   norm = (sum over tensors and elements of x^2)^(1/2)
 *   Y[i][j] = X[i][j] min(1, max_norm / (norm + eps))
 * The arrays dtypes, sizes, X and Y are host memory, read before the call
 * returns; the tensors are device memory.
 *   dtypes      type of each tensor and its result: SGEMM_F32, SGEMM_BF16, SGEMM_F16.
 *   sizes       elements of each, contiguous; 0 is allowed.
 *   Y           NULL: only the norm is formed (max_norm and eps are not used).
 *               Else each Y[i] is X[i] itself (in place; not written where
 *               the factor is 1) or overlaps no tensor of the list and no other result.  No
 *               two results overlap, so no tensor is in the list twice when
 *               it is scaled in place.
 *   norm        one float, or NULL.
 *   max_norm    >= 0; infinity scales nothing, whatever norm is not a NaN.      eps  >= 0.
 * The sum is held in 64 bits: values beyond 2^64 or below 2^-64 keep their
 * digits, and the norm is infinite only if it is beyond 3.4e38 or an element
 * is infinite.  An infinite norm gives the factor 0 (infinite elements become NaN) for a
 * finite max_norm, a NaN makes the norm and, scaled, every element NaN.  Where norm + eps
 * is 0 the factor is 1.
 * An empty list has norm 0.
 *   workspace   sgemm_clip_grad_norm_workspace_size(count, dtypes, sizes)
 *               bytes, 256-byte aligned.
 */
int sgemm_clip_grad_norm(int64_t count, const int *dtypes, const int64_t *sizes,
                         const void *const *X, void *const *Y, float max_norm, float eps,
                         float *norm, void *workspace, uint64_t workspace_bytes, void *stream);
uint64_t sgemm_clip_grad_norm_workspace_size(int64_t count, const int *dtypes,
                                             const int64_t *sizes);

#if defined(__GNUC__)
#pragma GCC visibility pop
#endif
#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_BLOCK_H */
