// C ABI of the layer operators: argument validation, the choice of kernel,
// workspace layout.  The contract is in include/sgemm_gb300_layers.h.
#include <cstdint>

#include <cuda_runtime.h>

#include "gemm_args.h"
#include "layers.h"
#include "layers_check.h"
#include "sgemm_gb300_layers.h"

namespace sgemm {

// Whether a product of M rows runs on the CUDA cores (linear_rows.cu), in one
// pass over the weights, or on the tensor cores.  Measured in a graph with the
// weights out of L2, in us, CUDA cores / tensor cores:
//   weights N x K    512x1024   1024x2048  1024x4096  1536x4096  2048x4096  4096x4096
//   bf16, 1 row      2.1 / 4.5  3.0 / 5.8  3.8 / 7.1  5.4 / 7.8  5.2 / 8.0  8.2 / 11.0
//   2 rows           2.2 / 4.4  3.0 / 5.7  3.9 / 7.1  6.0 / 7.8  5.4 / 8.0  8.4 / 11.2
//   4 rows           2.5 / 4.5  4.3 / 5.9  6.4 / 7.1  6.9 / 7.8  9.3 / 8.1  15.0 / 11.2
//   e4m3, 1 row      2.1 / 4.0  2.9 / 4.8  3.3 / 5.8  5.2 / 6.2  4.2 / 6.6  5.8 / 8.1
//   2 rows           2.2 / 4.0  2.8 / 4.8  4.4 / 5.9  5.4 / 6.3  6.3 / 6.7  9.0 / 8.3
// (4096 x 1024 much as 1024 x 4096.)  For the rows that the rule turns on, the sides
// come within 16 % of one another between 2^22 and 2^23 weights.  bf16 stored K x N,
// 4096 x 4096, 1 row: 24 / 11.  f32, whose planes the tensor cores need written
// first: 8 rows 25 / 48, 16 rows 45 / 48.
bool on_cuda_cores(int type, int64_t M, int64_t N, int64_t K, int transW) {
    if (K == 0) return true;
    if (type == SGEMM_F32) return M <= 16;
    if (!transW) return false;
    const int most = type == SGEMM_E4M3 ? 1 : 2;
    return M <= (N * K <= (1 << 22) ? 2 * most : most);
}

namespace {

size_t linear_bytes(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                    const void *W, int64_t ldw, int transW) {
    if (on_cuda_cores(dtype, M, N, K, transW)) return 0;
    if (dtype == SGEMM_F32)
        return f32_planes_bytes(M, K) + f32_planes_bytes(transW ? N : K, transW ? K : N);
    const int size = dtype_size(dtype);
    return copy_bytes(X, ldx, M, K, size) +
           copy_bytes(W, ldw, transW ? N : K, transW ? K : N, size);
}

// Layout of sgemm_linear_backward's workspace.
struct BackwardPlan {
    bool dz;                 // dZ is written (else dY is dZ)
    bool planes;             // f32: dZ is written as planes only, by the pass that forms it
    int64_t lddz;
    int parts;
    size_t dz_bytes, part_bytes, x_bytes, w_bytes, g_bytes;   // g: planes of dZ (f32)
    size_t total() const { return dz_bytes + part_bytes + x_bytes + w_bytes + g_bytes; }
};

BackwardPlan backward_plan(int dtype, int64_t M, int64_t N, int64_t K, const void *dY, int64_t lddy,
                           int act, const void *X, int64_t ldx, const void *W, int64_t ldw,
                           int transW, bool dx, bool dw, bool db) {
    BackwardPlan p = {};
    const int size = dtype_size(dtype);
    const bool f32 = dtype == SGEMM_F32;
    const bool dx_rows = on_cuda_cores(dtype, M, K, N, !transW);   // dX: any alignment
    const bool tc = (dx && !dx_rows) || dw;      // a tensor-core product reads dZ
    p.planes = f32 && K > 0 && tc && !(dx && dx_rows) && (act != SGEMM_ACT_NONE || db);
    p.dz = !p.planes && (dx || dw) && K > 0 &&
           (act != SGEMM_ACT_NONE || (!f32 && tc && !tma_ok(dY, lddy, size)));
    p.lddz = padded_ld(N, size);
    if (p.dz) p.dz_bytes = round256((size_t)M * p.lddz * size);
    p.parts = grad_parts(M, N);
    if (db) p.part_bytes = round256((size_t)p.parts * N * sizeof(float));
    if (K == 0) return p;
    if (f32) {
        if (dw) p.x_bytes = f32_planes_bytes(M, K);
        if (dx && !dx_rows) p.w_bytes = f32_planes_bytes(transW ? N : K, transW ? K : N);
        if (tc) p.g_bytes = f32_planes_bytes(M, N);
        return p;
    }
    if (dw) p.x_bytes = copy_bytes(X, ldx, M, K, size);
    if (dx && !dx_rows) p.w_bytes = copy_bytes(W, ldw, transW ? N : K, transW ? K : N, size);
    return p;
}

int linear(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
           const float *x_scale, const void *W, int64_t ldw, int transW, const float *w_scale,
           const void *bias, int activation, const void *residual, int64_t ldr, int out_dtype,
           void *Y, int64_t ldy, void *preact, int64_t ldp, void *workspace,
           uint64_t workspace_bytes, void *stream) {
    record_error(SGEMM_OK, "");
    const bool e4m3 = dtype == SGEMM_E4M3;
    if (!float_type(dtype) && !e4m3) return fail(SGEMM_EINVAL_TYPE, "dtype=%d", dtype);
    if (e4m3 ? out_dtype != SGEMM_BF16 && out_dtype != SGEMM_F16 : out_dtype != dtype)
        return fail(SGEMM_EINVAL_TYPE, "out_dtype=%d does not go with dtype=%d", out_dtype, dtype);
    if (activation < SGEMM_ACT_NONE || activation > SGEMM_ACT_SILU)
        return fail(SGEMM_EINVAL_TYPE, "activation=%d", activation);
    if ((transW != 0 && transW != 1) || (e4m3 && transW != 1))
        return fail(SGEMM_EINVAL_TRANS, "transW=%d: must be 0 or 1, and 1 for e4m3", transW);
    CHECK(check_sizes(M, N, K, "M, N, K"));
    if (M == 0 || N == 0) return SGEMM_OK;
    const int size = dtype_size(dtype), out = dtype_size(out_dtype);
    CHECK(check_matrix("X", X, ldx, K, size, K > 0));
    CHECK(check_matrix("W", W, ldw, transW ? K : N, size, K > 0));
    CHECK(check_matrix("Y", Y, ldy, N, out, true));
    CHECK(check_matrix("residual", residual, ldr, N, out, false));
    CHECK(check_matrix("preact", preact, ldp, N, out, false));
    if (residual == Y && ldr != ldy)
        return fail(SGEMM_EINVAL_LD, "residual is Y but ldr=%lld, ldy=%lld", (long long)ldr,
                    (long long)ldy);
    if (!aligned(bias, (uintptr_t)out)) return fail(SGEMM_EINVAL_PTR, "bias is not aligned");
    if (e4m3 != (x_scale != nullptr) || e4m3 != (w_scale != nullptr) || !aligned(x_scale, 4) ||
        !aligned(w_scale, 4))
        return fail(SGEMM_EINVAL_PTR, "x_scale and w_scale are required for e4m3, 4-byte aligned, "
                    "and NULL for the other types");
    const size_t need = linear_bytes(dtype, M, N, K, X, ldx, W, ldw, transW);
    CHECK(check_workspace(workspace, workspace_bytes, need));
    CHECK(require_device());
    LayerEpi epi = {Y, preact, residual, bias, x_scale, w_scale, ldy, ldp, ldr, (int)M, (int)N,
                    activation, out_dtype, 1};
    if (K == 0) epi.sx = epi.sw = nullptr;   // an empty sum is 0 in any unit, a NaN's too
    epi.vec = vector_width(out_dtype, epi);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (on_cuda_cores(dtype, M, N, K, transW))
        return launched(launch_linear_rows(dtype, X, ldx, W, ldw, K > 0 ? transW : 1, (int)K, epi,
                                           s));
    if (dtype == SGEMM_F32) {
        const int64_t wr = transW ? N : K, wc = transW ? K : N;
        char *const wsw = static_cast<char *>(workspace) + f32_planes_bytes(M, K);
        const F32Operand in[2] = {{static_cast<const float *>(X), ldx, M, K, workspace},
                                  {static_cast<const float *>(W), ldw, wr, wc, wsw}};
        const cudaError_t split = launch_f32_split(in, 2, 0, s);
        if (split != cudaSuccess) return launched(split);
        return launched(launch_linear_f32({workspace, M, K, true}, {wsw, wr, wc, transW != 0},
                                          (int)K, epi, 0, s));
    }
    char *ws = static_cast<char *>(workspace);
    cudaError_t e = place(X, ldx, M, K, size, ws, s);
    if (e == cudaSuccess) e = place(W, ldw, transW ? N : K, transW ? K : N, size, ws, s);
    if (e != cudaSuccess) return launched(e);
    return launched(launch_linear_tc(dtype, {X, ldx, true}, {W, ldw, transW != 0}, (int)K, epi, 0,
                                     s));
}

int linear_backward(int dtype, int64_t M, int64_t N, int64_t K, const void *dY, int64_t lddy,
                    const void *Z, int64_t ldz, int activation, const void *X, int64_t ldx,
                    const void *W, int64_t ldw, int transW, void *dX, int64_t lddx, void *dW,
                    int64_t lddw, void *db, void *workspace, uint64_t workspace_bytes,
                    void *stream) {
    record_error(SGEMM_OK, "");
    if (!float_type(dtype)) return fail(SGEMM_EINVAL_TYPE, "dtype=%d", dtype);
    if (activation < SGEMM_ACT_NONE || activation > SGEMM_ACT_SILU)
        return fail(SGEMM_EINVAL_TYPE, "activation=%d", activation);
    if (transW != 0 && transW != 1) return fail(SGEMM_EINVAL_TRANS, "transW=%d", transW);
    CHECK(check_sizes(M, N, K, "M, N, K"));
    const int size = dtype_size(dtype);
    const bool dx = dX != nullptr && M > 0 && K > 0;
    const bool dw = dW != nullptr && N > 0 && K > 0;
    const bool dbias = db != nullptr && N > 0;
    const int64_t wrows = transW ? N : K, wcols = transW ? K : N;
    const bool work = M > 0 && N > 0;
    CHECK(check_matrix("dX", dX, lddx, K, size, false));
    CHECK(check_matrix("dW", dW, lddw, wcols, size, false));
    if (!aligned(db, (uintptr_t)size)) return fail(SGEMM_EINVAL_PTR, "db is not aligned");
    if (!dx && !dw && !dbias) return SGEMM_OK;
    CHECK(check_matrix("dY", dY, lddy, N, size, work));
    CHECK(check_matrix("Z", Z, ldz, N, size, work && activation != SGEMM_ACT_NONE));
    CHECK(check_matrix("X", X, ldx, K, size, work && dw));
    CHECK(check_matrix("W", W, ldw, wcols, size, work && dx));
    BackwardPlan p = {};
    if (work) {
        p = backward_plan(dtype, M, N, K, dY, lddy, activation, X, ldx, W, ldw, transW, dx, dw,
                          dbias);
        CHECK(check_workspace(workspace, workspace_bytes, p.total()));
    }
    CHECK(require_device());
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (!work) {   // empty sums
        if (dx) e = cudaMemset2DAsync(dX, lddx * size, 0, K * size, M, s);
        if (dw && e == cudaSuccess) e = cudaMemset2DAsync(dW, lddw * size, 0, wcols * size, wrows, s);
        if (dbias && e == cudaSuccess) e = cudaMemsetAsync(db, 0, N * size, s);
        return launched(e);
    }
    char *ws = static_cast<char *>(workspace);
    void *dZ = p.dz ? ws : nullptr;
    ws += p.dz_bytes;
    float *partial = dbias ? reinterpret_cast<float *>(ws) : nullptr;
    ws += p.part_bytes;
    char *const wsx = ws, *const wsw = wsx + p.x_bytes, *const wsg = wsw + p.w_bytes;   // f32
    const bool dx_rows = on_cuda_cores(dtype, M, K, N, !transW);
    const bool tdx = dx && !dx_rows;
    // what does not wait for what: the planes of X and W for the pass over dZ, the
    // two products and, behind a product, the bias gradient's last sum (500 x 777 x
    // 1001 f32: 31.5 us with every launch after the one before it, 22.8 so; 512 x
    // 1024 x 1024 bf16 14.3 and 11.9)
    const int split_at = p.planes ? kChainPrev : 0;
    const bool sum_last = tdx || dw;
    if (p.dz || p.planes || dbias)
        e = launch_linear_dz(dtype, dY, lddy, Z, ldz, activation, (int)M, (int)N,
                             p.planes ? wsg : dZ, p.planes ? f32_plane_ld(N) : p.lddz,
                             p.planes ? M * f32_plane_ld(N) : 0, partial,
                             p.planes ? kChainNext : 0, s);
    if (dbias && !sum_last && e == cudaSuccess)
        e = launch_column_sum(dtype, partial, p.parts, N, db, 0, s);
    if (e != cudaSuccess) return launched(e);
    const void *g = p.dz ? dZ : dY;
    const int64_t ldg = p.dz ? p.lddz : lddy;
    if (dx && dx_rows)
        // reduction over the output features: W's other orientation
        e = launch_linear_rows(dtype, g, ldg, W, ldw, !transW, (int)N,
                               plain_epi(dtype, dX, lddx, M, K), s);
    if (e != cudaSuccess) return launched(e);
    int before = dw || dbias ? kChainNext : 0;
    int after = (tdx ? kChainPrev : 0) | (dbias ? kChainNext : 0);
    if (tdx && dw) {
        const ProductSize a = {(int)M, (int)K, (int)N}, b = {(int)wrows, (int)wcols, (int)M};
        if (dtype == SGEMM_F32 ? linear_f32_side_by_side(a, b)
                               : linear_tc_side_by_side(dtype, a, b)) {
            before |= kChainHalf;
            after |= kChainHalf;
        }
    }
    if (dtype == SGEMM_F32) {
        // planes of dZ (for both products), X and W, two matrices a launch
        F32Operand in[3];
        int count = 0;
        if (dw) in[count++] = {static_cast<const float *>(X), ldx, M, K, wsx};
        if (tdx) in[count++] = {static_cast<const float *>(W), ldw, wrows, wcols, wsw};
        if (!p.planes && (tdx || dw)) in[count++] = {static_cast<const float *>(g), ldg, M, N, wsg};
        for (int i = 0; i < count && e == cudaSuccess; i += 2)
            e = launch_f32_split(in + i, count - i < 2 ? count - i : 2, split_at, s);
        if (tdx && e == cudaSuccess)
            e = launch_linear_f32({wsg, M, N, true}, {wsw, wrows, wcols, transW == 0}, (int)N,
                                  plain_epi(dtype, dX, lddx, M, K), before, s);
        if (dw && e == cudaSuccess) {
            const F32Planes Gp = {wsg, M, N, false}, Xp = {wsx, M, K, false};
            e = launch_linear_f32(transW ? Gp : Xp, transW ? Xp : Gp, (int)M,
                                  plain_epi(dtype, dW, lddw, wrows, wcols), after, s);
        }
        if (dbias && sum_last && e == cudaSuccess)
            e = launch_column_sum(dtype, partial, p.parts, N, db, kChainPrev, s);
        return launched(e);
    }
    if (tdx) e = place(W, ldw, wrows, wcols, size, ws, s);
    if (dw && e == cudaSuccess) e = place(X, ldx, M, K, size, ws, s);
    if (tdx && e == cudaSuccess)
        e = launch_linear_tc(dtype, {g, ldg, true}, {W, ldw, transW == 0}, (int)N,
                             plain_epi(dtype, dX, lddx, M, K), before, s);
    if (dw && e == cudaSuccess) {
        const TcOperand G = {g, ldg, false}, Xo = {X, ldx, false};
        e = launch_linear_tc(dtype, transW ? G : Xo, transW ? Xo : G, (int)M,
                             plain_epi(dtype, dW, lddw, wrows, wcols), after, s);
    }
    if (dbias && sum_last && e == cudaSuccess)
        e = launch_column_sum(dtype, partial, p.parts, N, db, kChainPrev, s);
    return launched(e);
}

int check_norm(int dtype, int64_t rows, int64_t D) {
    record_error(SGEMM_OK, "");
    if (!float_type(dtype)) return fail(SGEMM_EINVAL_TYPE, "dtype=%d", dtype);
    return check_sizes(rows, D, 0, "rows, D");
}

}  // namespace
}  // namespace sgemm

extern "C" {

int sgemm_linear(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                 const float *x_scale, const void *W, int64_t ldw, int transW, const float *w_scale,
                 const void *bias, int activation, const void *residual, int64_t ldr, int out_dtype,
                 void *Y, int64_t ldy, void *preact, int64_t ldp, void *workspace,
                 uint64_t workspace_bytes, void *stream) {
    return sgemm::linear(dtype, M, N, K, X, ldx, x_scale, W, ldw, transW, w_scale, bias, activation,
                         residual, ldr, out_dtype, Y, ldy, preact, ldp, workspace, workspace_bytes,
                         stream);
}

uint64_t sgemm_linear_workspace_size(int dtype, int64_t M, int64_t N, int64_t K, const void *X,
                                     int64_t ldx, const void *W, int64_t ldw, int transW) {
    if (M <= 0 || N <= 0 || K <= 0 || dtype < SGEMM_F32 || dtype > SGEMM_E4M3) return 0;
    return sgemm::linear_bytes(dtype, M, N, K, X, ldx, W, ldw, transW);
}

int sgemm_linear_backward(int dtype, int64_t M, int64_t N, int64_t K, const void *dY, int64_t lddy,
                          const void *Z, int64_t ldz, int activation, const void *X, int64_t ldx,
                          const void *W, int64_t ldw, int transW, void *dX, int64_t lddx, void *dW,
                          int64_t lddw, void *db, void *workspace, uint64_t workspace_bytes,
                          void *stream) {
    return sgemm::linear_backward(dtype, M, N, K, dY, lddy, Z, ldz, activation, X, ldx, W, ldw,
                                  transW, dX, lddx, dW, lddw, db, workspace, workspace_bytes,
                                  stream);
}

uint64_t sgemm_linear_backward_workspace_size(int dtype, int64_t M, int64_t N, int64_t K,
                                              const void *dY, int64_t lddy, int activation,
                                              const void *X, int64_t ldx, const void *W,
                                              int64_t ldw, int transW) {
    if (M <= 0 || N <= 0 || K < 0 || !sgemm::float_type(dtype)) return 0;
    return sgemm::backward_plan(dtype, M, N, K, dY, lddy, activation, X, ldx, W, ldw, transW, true,
                                true, true)
        .total();
}

int sgemm_add_rmsnorm(int dtype, int64_t rows, int64_t D, const void *X, int64_t ldx,
                      const void *residual, int64_t ldr, const void *weight, float eps, void *S,
                      int64_t lds, void *Y, int64_t ldy, float *q_scale, float *rstd, void *stream) {
    using namespace sgemm;
    CHECK(check_norm(dtype, rows, D));
    // (rows of no elements have a scale and a reciprocal root all the same)
    if (rows == 0 || (D == 0 && q_scale == nullptr && rstd == nullptr)) return SGEMM_OK;
    const int size = dtype_size(dtype);
    CHECK(check_matrix("X", X, ldx, D, size, D > 0));
    CHECK(check_matrix("residual", residual, ldr, D, size, false));
    CHECK(check_matrix("S", S, lds, D, size, false));
    CHECK(check_matrix("Y", Y, ldy, D, q_scale != nullptr ? 1 : size, D > 0));
    CHECK(check_matrix("weight", weight, D > 1 ? D : 1, D, size, D > 0));
    if (!aligned(q_scale, 4) || !aligned(rstd, 4))
        return fail(SGEMM_EINVAL_PTR, "q_scale or rstd is not 4-byte aligned");
    CHECK(require_device());
    return launched(launch_add_rmsnorm(dtype, rows, D, X, ldx, residual, ldr, weight, eps, S, lds, Y,
                                       ldy, q_scale, rstd, static_cast<cudaStream_t>(stream)));
}

int sgemm_add_rmsnorm_backward(int dtype, int64_t rows, int64_t D, const void *dY, int64_t lddy,
                               const void *S, int64_t lds, const float *rstd, const void *weight,
                               const void *dS, int64_t ldds, void *dX, int64_t lddx, void *dweight,
                               void *workspace, uint64_t workspace_bytes, void *stream) {
    using namespace sgemm;
    CHECK(check_norm(dtype, rows, D));
    if (D == 0) return SGEMM_OK;
    const int size = dtype_size(dtype);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!aligned(dweight, (uintptr_t)size)) return fail(SGEMM_EINVAL_PTR, "dweight is not aligned");
    if (rows == 0) {   // an empty sum
        if (dweight == nullptr) return SGEMM_OK;
        CHECK(require_device());
        return launched(cudaMemsetAsync(dweight, 0, D * size, s));
    }
    CHECK(check_matrix("dY", dY, lddy, D, size, true));
    CHECK(check_matrix("S", S, lds, D, size, true));
    CHECK(check_matrix("weight", weight, D, D, size, true));
    CHECK(check_matrix("rstd", rstd, 1, 1, 4, true));
    CHECK(check_matrix("dS", dS, ldds, D, size, false));
    CHECK(check_matrix("dX", dX, lddx, D, size, true));
    if (dweight != nullptr)
        CHECK(check_workspace(workspace, workspace_bytes,
                              sgemm_add_rmsnorm_backward_workspace_size(dtype, rows, D)));
    CHECK(require_device());
    return launched(launch_add_rmsnorm_backward(dtype, rows, D, dY, lddy, S, lds, rstd, weight, dS,
                                                ldds, dX, lddx, dweight,
                                                static_cast<float *>(workspace), s));
}

uint64_t sgemm_add_rmsnorm_backward_workspace_size(int dtype, int64_t rows, int64_t D) {
    if (rows <= 0 || D <= 0 || !sgemm::float_type(dtype)) return 0;
    return (uint64_t)sgemm::rmsnorm_backward_parts(dtype, rows, D) * (uint64_t)D * sizeof(float);
}

int sgemm_quantize_rows(int dtype, int64_t rows, int64_t D, const void *X, int64_t ldx, void *Q,
                        int64_t ldq, float *scale, void *stream) {
    using namespace sgemm;
    CHECK(check_norm(dtype, rows, D));
    if (rows == 0) return SGEMM_OK;
    CHECK(check_matrix("X", X, ldx, D, dtype_size(dtype), D > 0));
    CHECK(check_matrix("Q", Q, ldq, D, 1, D > 0));
    CHECK(check_matrix("scale", scale, 1, 1, 4, true));
    CHECK(require_device());
    return launched(launch_quantize_rows(dtype, rows, D, X, ldx, Q, ldq, scale,
                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
