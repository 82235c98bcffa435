// C ABI of the gated feed-forward block's operators: argument validation, the choice of
// kernel, workspace layout.  The contract is in include/sgemm_gb300_block.h.
#include <algorithm>
#include <cstdint>
#include <exception>
#include <vector>

#include <cuda_runtime.h>

#include "layers.h"
#include "layers_check.h"
#include "sgemm_gb300_block.h"

namespace sgemm {
namespace {

// The gated product of few rows on the CUDA cores, where its tiles on the tensor cores
// take longer; us there / here, weights of both out of L2 (features x K):
//   bf16   11264 x 4096  1 row 31.0 / 30.9, 2 rows 37.0 / 30.8; 4096 x 4096  2 rows 14.3 / 14.9, 4 rows
//          25.2 / 14.8; 2048 x 2048  4 rows 7.1 / 8.3, 6 rows 10.2 / 8.2; 2048 x 1024  6 rows 6.4 / 6.8
//   e4m3   11264 x 4096  1 row 21.7 / 19.4; 4096 x 4096  1 row 9.3 / 10.7, 2 rows 14.5 / 10.5; 2048 x
//          2048  2 rows 5.1 / 6.8, 3 rows 6.8 / 6.7; 2048 x 1024  3 rows 5.3 / 5.9
//   f32    11264 x 4096  4 rows 286 / 76, 8 rows 286 / 106, 16 rows 286 / 212; 4096 x 4096  8 rows 91 / 44,
//          16 rows 91 / 90, 24 rows 91 / 128; 2048 x 2048  16 rows 24.9 / 21.3; 1024 x 1024  16 rows
//          11.8 / 7.6; 300 x 333  16 rows 9.4 / 5.8
//   f32 stored K x N   11264 x 4096  1 row 285 / 55, 8 rows 284 / 127, 16 rows 285 / 241; 4096 x 4096
//          1 row 93 / 23, 16 rows 93 / 68; 2048 x 2048  8 rows 24.8 / 23.9, 16 rows 25.0 / 20.0;
//          1024 x 1024  16 rows 12.7 / 13.0; 300 x 333  16 rows 9.5 / 6.5
bool gated_on_cuda_cores(int type, int64_t M, int64_t N, int64_t K, int transW) {
    if (K == 0) return true;
    const int64_t weights = 2 * N * K;
    if (type == SGEMM_F32) return M <= 16;
    if (!transW) return false;
    if (type == SGEMM_E4M3)
        return M <= (weights <= 1 << 22 ? 4 : weights <= 1 << 23 ? 2 : weights <= 1 << 25 ? 1 : 0);
    return M <= (weights <= 1 << 22 ? 8 : weights <= 1 << 23 ? 4 : weights <= 1 << 24 ? 2 : 1);
}

size_t gated_bytes(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                   const void *Wg, int64_t ldwg, const void *Wu, int64_t ldwu, int transW) {
    if (gated_on_cuda_cores(dtype, M, N, K, transW)) return 0;
    const int64_t wr = transW ? N : K, wc = transW ? K : N;
    if (dtype == SGEMM_F32) return f32_planes_bytes(M, K) + 2 * f32_planes_bytes(wr, wc);
    const int size = dtype_size(dtype);
    return copy_bytes(X, ldx, M, K, size) + copy_bytes(Wg, ldwg, wr, wc, size) +
           copy_bytes(Wu, ldwu, wr, wc, size);
}

int gated_vector_width(int type, const GatedEpi &e) {
    const int size = dtype_size(type);
    auto all = [&](int n) {
        const uintptr_t bytes = (uintptr_t)(n * size);
        auto matrix = [&](const void *p, int64_t ld) {
            return p == nullptr || (aligned(p, bytes) && ld % n == 0);
        };
        return matrix(e.H, e.ldh) && matrix(e.Zg, e.ldg) && matrix(e.Zu, e.ldu) &&
               aligned(e.bg, bytes) && aligned(e.bu, bytes) && aligned(e.sg, n == 8 ? 16 : 4) &&
               aligned(e.su, n == 8 ? 16 : 4);
    };
    return size == 2 && all(8) ? 8 : all(4) ? 4 : size == 2 && all(2) ? 2 : 1;
}

// Operands that TMA cannot read where they lie, copied to the workspace in one launch.
class Placing {
public:
    Placing(char *ws, int size) : ws_(ws), size_(size) {}
    void add(const void *&p, int64_t &ld, int64_t rows, int64_t cols) {
        if (tma_ok(p, ld, size_)) return;
        const int64_t to = padded_ld(cols, size_);
        jobs_[count_++] = {p, ws_, ld * size_, to * size_, rows, cols * size_, 0};
        p = ws_;
        ld = to;
        ws_ += round256((size_t)rows * to * size_);
    }
    cudaError_t run(cudaStream_t s) {
        return count_ > 0 ? launch_repack3(jobs_, count_, s) : cudaSuccess;
    }

private:
    RepackJob jobs_[3];
    int count_ = 0;
    char *ws_;
    int size_;
};

int check_gated_sizes(int64_t M, int64_t N, int64_t K) {
    CHECK(check_sizes(M, N, K, "M, N, K"));
    if (N > kMaxDim / 2)
        return fail(SGEMM_EINVAL_DIM, "N = %lld: a gated layer takes up to 2^29 features",
                    (long long)N);
    return SGEMM_OK;
}

int gated_linear(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                 const float *x_scale, const void *Wg, int64_t ldwg, const float *gate_scale,
                 const void *Wu, int64_t ldwu, const float *up_scale, int transW,
                 const void *bias_gate, const void *bias_up, int activation, int out_dtype, void *H,
                 int64_t ldh, void *preact_gate, int64_t ldpg, void *preact_up, int64_t ldpu,
                 void *workspace, uint64_t workspace_bytes, cudaStream_t s) {
    record_error(SGEMM_OK, "");
    const bool e4m3 = dtype == SGEMM_E4M3;
    if (!float_type(dtype) && !e4m3) return fail(SGEMM_EINVAL_TYPE, "dtype=%d", dtype);
    if (e4m3 ? out_dtype != SGEMM_BF16 && out_dtype != SGEMM_F16 : out_dtype != dtype)
        return fail(SGEMM_EINVAL_TYPE, "out_dtype=%d does not go with dtype=%d", out_dtype, dtype);
    if (activation < SGEMM_ACT_NONE || activation > SGEMM_ACT_SILU)
        return fail(SGEMM_EINVAL_TYPE, "activation=%d", activation);
    if ((transW != 0 && transW != 1) || (e4m3 && transW != 1))
        return fail(SGEMM_EINVAL_TRANS, "transW=%d: must be 0 or 1, and 1 for e4m3", transW);
    CHECK(check_gated_sizes(M, N, K));
    if (M == 0 || N == 0) return SGEMM_OK;
    const int size = dtype_size(dtype), out = dtype_size(out_dtype);
    const int64_t wr = transW ? N : K, wc = transW ? K : N;
    CHECK(check_matrix("X", X, ldx, K, size, K > 0));
    CHECK(check_matrix("Wg", Wg, ldwg, wc, size, K > 0));
    CHECK(check_matrix("Wu", Wu, ldwu, wc, size, K > 0));
    CHECK(check_matrix("H", H, ldh, N, out, true));
    CHECK(check_matrix("preact_gate", preact_gate, ldpg, N, out, false));
    CHECK(check_matrix("preact_up", preact_up, ldpu, N, out, false));
    if (!aligned(bias_gate, (uintptr_t)out) || !aligned(bias_up, (uintptr_t)out))
        return fail(SGEMM_EINVAL_PTR, "a bias is not aligned");
    for (const float *scale : {x_scale, gate_scale, up_scale})
        if (e4m3 != (scale != nullptr) || !aligned(scale, 4))
            return fail(SGEMM_EINVAL_PTR, "x_scale, gate_scale and up_scale are required for e4m3, "
                        "4-byte aligned, and NULL for the other types");
    const size_t need = gated_bytes(dtype, M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, transW);
    CHECK(check_workspace(workspace, workspace_bytes, need));
    CHECK(require_device());
    GatedEpi epi = {H,    preact_gate, preact_up, bias_gate, bias_up, x_scale,    gate_scale, up_scale,
                    ldh,  ldpg,        ldpu,      (int)M,    (int)N,  activation, out_dtype,  1};
    if (K == 0) epi.sx = epi.sg = epi.su = nullptr;   // an empty sum is 0 in any unit
    epi.vec = gated_vector_width(out_dtype, epi);
    if (gated_on_cuda_cores(dtype, M, N, K, transW))
        return launched(launch_gated_rows(dtype, X, ldx, Wg, ldwg, Wu, ldwu, K == 0 ? 1 : transW,
                                          (int)K, epi, s));   // (K == 0: no weight is read)
    char *ws = static_cast<char *>(workspace);
    if (dtype == SGEMM_F32) {
        char *const wsg = ws + f32_planes_bytes(M, K), *const wsu = wsg + f32_planes_bytes(wr, wc);
        const F32Operand in[3] = {{static_cast<const float *>(X), ldx, M, K, ws},
                                  {static_cast<const float *>(Wg), ldwg, wr, wc, wsg},
                                  {static_cast<const float *>(Wu), ldwu, wr, wc, wsu}};
        const cudaError_t split = launch_f32_split(in, 3, 0, s);
        if (split != cudaSuccess) return launched(split);
        return launched(launch_gated_f32({ws, M, K, true}, {wsg, wr, wc, transW != 0},
                                         {wsu, wr, wc, transW != 0}, (int)K, epi, s));
    }
    Placing placing(ws, size);
    placing.add(X, ldx, M, K);
    placing.add(Wg, ldwg, wr, wc);
    placing.add(Wu, ldwu, wr, wc);
    const cudaError_t e = placing.run(s);
    if (e != cudaSuccess) return launched(e);
    return launched(launch_gated_tc(dtype, {X, ldx, true}, {Wg, ldwg, transW != 0},
                                    {Wu, ldwu, transW != 0}, (int)K, epi, s));
}

// Layout of sgemm_gated_linear_backward's workspace: both dZ (f32: as planes), the partial
// column sums, then X and the weights (f32: their planes) where they are needed.
struct GatedBackward {
    int64_t lddz;
    int parts;
    size_t dz_bytes, part_bytes, x_bytes, g_bytes, u_bytes;   // dz_bytes: of one of the two
    size_t total() const { return 2 * dz_bytes + part_bytes + x_bytes + g_bytes + u_bytes; }
};

GatedBackward gated_backward_plan(int dtype, int64_t M, int64_t N, int64_t K, const void *X,
                                  int64_t ldx, const void *Wg, int64_t ldwg, const void *Wu,
                                  int64_t ldwu, int transW, bool dx, bool dw, bool db) {
    GatedBackward p = {};
    const int size = dtype_size(dtype);
    const int64_t wr = transW ? N : K, wc = transW ? K : N;
    p.parts = gated_parts(dtype, M, N);
    if (db) p.part_bytes = round256((size_t)p.parts * 2 * N * sizeof(float));
    if (K == 0) return p;
    if (dtype == SGEMM_F32) {
        p.lddz = f32_plane_ld(N);
        if (dx || dw) p.dz_bytes = f32_planes_bytes(M, N);
        if (dw) p.x_bytes = f32_planes_bytes(M, K);
        if (dx) p.g_bytes = p.u_bytes = f32_planes_bytes(wr, wc);
        return p;
    }
    p.lddz = padded_ld(N, size);
    if (dx || dw) p.dz_bytes = round256((size_t)M * p.lddz * size);
    if (dw) p.x_bytes = copy_bytes(X, ldx, M, K, size);
    if (dx) p.g_bytes = copy_bytes(Wg, ldwg, wr, wc, size);
    if (dx) p.u_bytes = copy_bytes(Wu, ldwu, wr, wc, size);
    return p;
}

int gated_linear_backward(int dtype, int64_t M, int64_t N, int64_t K, const void *dH, int64_t lddh,
                          const void *Zg, int64_t ldzg, const void *Zu, int64_t ldzu, int activation,
                          const void *X, int64_t ldx, const void *Wg, int64_t ldwg, const void *Wu,
                          int64_t ldwu, int transW, void *dX, int64_t lddx, void *dWg,
                          int64_t lddwg, void *dWu, int64_t lddwu, void *db_gate, void *db_up,
                          void *workspace, uint64_t workspace_bytes, cudaStream_t s) {
    record_error(SGEMM_OK, "");
    if (!float_type(dtype)) return fail(SGEMM_EINVAL_TYPE, "dtype=%d", dtype);
    if (activation < SGEMM_ACT_NONE || activation > SGEMM_ACT_SILU)
        return fail(SGEMM_EINVAL_TYPE, "activation=%d", activation);
    if (transW != 0 && transW != 1) return fail(SGEMM_EINVAL_TRANS, "transW=%d", transW);
    CHECK(check_gated_sizes(M, N, K));
    const int size = dtype_size(dtype);
    const int64_t wr = transW ? N : K, wc = transW ? K : N;
    const bool dx = dX != nullptr && M > 0 && K > 0;
    const bool dwg = dWg != nullptr && N > 0 && K > 0, dwu = dWu != nullptr && N > 0 && K > 0;
    const bool db = (db_gate != nullptr || db_up != nullptr) && N > 0;
    const bool work = M > 0 && N > 0, dw = dwg || dwu;
    CHECK(check_matrix("dX", dX, lddx, K, size, false));
    CHECK(check_matrix("dWg", dWg, lddwg, wc, size, false));
    CHECK(check_matrix("dWu", dWu, lddwu, wc, size, false));
    if (!aligned(db_gate, (uintptr_t)size) || !aligned(db_up, (uintptr_t)size))
        return fail(SGEMM_EINVAL_PTR, "db_gate or db_up is not aligned");
    if (!dx && !dw && !db) return SGEMM_OK;
    CHECK(check_matrix("dH", dH, lddh, N, size, work));
    CHECK(check_matrix("Zg", Zg, ldzg, N, size, work));
    CHECK(check_matrix("Zu", Zu, ldzu, N, size, work));
    CHECK(check_matrix("X", X, ldx, K, size, work && dw));
    CHECK(check_matrix("Wg", Wg, ldwg, wc, size, work && dx));
    CHECK(check_matrix("Wu", Wu, ldwu, wc, size, work && dx));
    GatedBackward p = {};
    if (work) {
        p = gated_backward_plan(dtype, M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, transW, dx, dw, db);
        CHECK(check_workspace(workspace, workspace_bytes, p.total()));
    }
    CHECK(require_device());
    cudaError_t e = cudaSuccess;
    if (!work) {   // empty sums
        if (dx) e = cudaMemset2DAsync(dX, lddx * size, 0, K * size, M, s);
        if (dwg && e == cudaSuccess) e = cudaMemset2DAsync(dWg, lddwg * size, 0, wc * size, wr, s);
        if (dwu && e == cudaSuccess) e = cudaMemset2DAsync(dWu, lddwu * size, 0, wc * size, wr, s);
        for (void *d : {db_gate, db_up})
            if (d != nullptr && e == cudaSuccess) e = cudaMemsetAsync(d, 0, N * size, s);
        return launched(e);
    }
    const bool f32 = dtype == SGEMM_F32, products = dx || dw;
    char *ws = static_cast<char *>(workspace);
    void *const zg = products ? ws : nullptr, *const zu = products ? ws + p.dz_bytes : nullptr;
    ws += 2 * p.dz_bytes;
    float *const partial = db ? reinterpret_cast<float *>(ws) : nullptr;
    ws += p.part_bytes;
    // What reads nothing of one another overlaps (kChainPrev, kChainNext): in f32 the planes of X
    // and the weights with the pass over dH, then the three products and the biases' last sum.
    e = launch_gated_dz(dtype, dH, lddh, Zg, ldzg, Zu, ldzu, activation, (int)M, (int)N, zg, zu,
                        p.lddz, f32 ? M * p.lddz : 0, partial, f32 && products ? kChainNext : 0, s);
    if (e != cudaSuccess) return launched(e);
    char *const wsx = ws, *const wsg = wsx + p.x_bytes, *const wsu = wsg + p.g_bytes;   // f32
    if (f32 && products) {
        F32Operand in[3];
        int count = 0;
        if (dw) in[count++] = {static_cast<const float *>(X), ldx, M, K, wsx};
        if (dx) in[count++] = {static_cast<const float *>(Wg), ldwg, wr, wc, wsg};
        if (dx) in[count++] = {static_cast<const float *>(Wu), ldwu, wr, wc, wsu};
        e = launch_f32_split(in, count, kChainPrev, s);
    } else if (products) {
        Placing placing(ws, size);
        if (dw) placing.add(X, ldx, M, K);
        if (dx) placing.add(Wg, ldwg, wr, wc);
        if (dx) placing.add(Wu, ldwu, wr, wc);
        e = placing.run(s);
    }
    // dX has all SMs, the weights' gradients, which read the same X, half of them each where that
    // is no slower.  Large products: the weights' first (gradients of 2048 x 5632 x 2048 bf16 136.4 ->
    // 132.8 us, 1000 x 1376 x 1008 f32 77.4 -> 74.3); small ones: dX first (300^3 bf16 11.0, else 12.3;
    // 512 x 1280 x 236 f32 21.9, else 29.0).
    const int half =
        dwg && dwu && gated_side_by_side(dtype, {(int)wr, (int)wc, (int)M}) ? kChainHalf : 0;
    const bool weights_first = (double)M * N * K >= (double)(1 << 30);
    int left = (int)dx + (int)dwg + (int)dwu + (int)db, done = 0;
    auto place_in_chain = [&] {
        --left;
        return (done++ > 0 ? kChainPrev : 0) | (left > 0 ? kChainNext : 0);
    };
    auto input_gradient = [&] {
        if (!dx || e != cudaSuccess) return;
        const LayerEpi epi = plain_epi(dtype, dX, lddx, M, K);
        const int at = place_in_chain();
        if (f32)
            e = launch_sum_f32({{zg, M, N, true}, {zu, M, N, true}},
                               {{wsg, wr, wc, transW == 0}, {wsu, wr, wc, transW == 0}}, (int)N, epi,
                               at, s);
        else
            e = launch_sum_tc(dtype, {{zg, p.lddz, true}, {zu, p.lddz, true}},
                              {{Wg, ldwg, transW == 0}, {Wu, ldwu, transW == 0}}, 2, (int)N, epi, at,
                              s);
    };
    auto weight_gradients = [&] {
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
            if (!(i == 0 ? dwg : dwu)) continue;
            const LayerEpi epi = plain_epi(dtype, i == 0 ? dWg : dWu, i == 0 ? lddwg : lddwu, wr, wc);
            const void *z = i == 0 ? zg : zu;
            const int at = place_in_chain() | half;
            if (f32) {
                const F32Planes G = {z, M, N, false}, Xp = {wsx, M, K, false};
                e = launch_linear_f32(transW ? G : Xp, transW ? Xp : G, (int)M, epi, at, s);
            } else {
                const TcOperand G = {z, p.lddz, false}, Xo = {X, ldx, false};
                const TcOperand &A = transW ? G : Xo, &B = transW ? Xo : G;
                e = launch_sum_tc(dtype, {A, A}, {B, B}, 1, (int)M, epi, at, s);
            }
        }
    };
    if (weights_first) weight_gradients();
    input_gradient();
    if (!weights_first) weight_gradients();
    if (db && e == cudaSuccess)
        e = launch_column_sum2(dtype, partial, p.parts, N, db_gate, db_up, place_in_chain(), s);
    return launched(e);
}

int check_norm(int dtype, int64_t rows, int64_t D) {
    record_error(SGEMM_OK, "");
    if (!float_type(dtype)) return fail(SGEMM_EINVAL_TYPE, "dtype=%d", dtype);
    return check_sizes(rows, D, 0, "rows, D");
}

// Whether a result overlaps a tensor other than its own or another result.  Both lists'
// ranges in order of their addresses (as tensors of one buffer come), then one walk over both.
bool results_overlap(int64_t count, const int *dtypes, const int64_t *sizes, const void *const *X,
                     void *const *Y) {
    struct Range {
        uintptr_t begin, end;
    };
    std::vector<Range> in, out;   // in: tensors that are not scaled in place
    in.reserve((size_t)count);
    out.reserve((size_t)count);
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t bytes = (uintptr_t)sizes[i] * dtype_size(dtypes[i]);
        const uintptr_t x = reinterpret_cast<uintptr_t>(X[i]), y = reinterpret_cast<uintptr_t>(Y[i]);
        if (x != y) in.push_back({x, x + bytes});
        out.push_back({y, y + bytes});
    }
    const auto before = [](const Range &a, const Range &b) { return a.begin < b.begin; };
    for (std::vector<Range> *r : {&in, &out})
        if (!std::is_sorted(r->begin(), r->end(), before)) std::sort(r->begin(), r->end(), before);
    uintptr_t results = 0, all = 0;   // where those so far end
    auto i = in.begin();
    for (auto o = out.begin(); o != out.end() || i != in.end();) {
        const bool result = i == in.end() || (o != out.end() && o->begin < i->begin);
        const Range a = result ? *o++ : *i++;
        if (a.begin < (result ? all : results)) return true;
        all = std::max(all, a.end);
        if (result) results = std::max(results, a.end);
    }
    return false;
}

int clip_grad_norm(int64_t count, const int *dtypes, const int64_t *sizes, const void *const *X,
                   void *const *Y, float max_norm, float eps, float *norm, void *workspace,
                   uint64_t workspace_bytes, cudaStream_t s) {
    record_error(SGEMM_OK, "");
    if (count < 0 || count > kMaxDim)
        return fail(SGEMM_EINVAL_DIM, "count = %lld: must be 0 .. 2^30", (long long)count);
    if (count > 0 && (dtypes == nullptr || sizes == nullptr || X == nullptr))
        return fail(SGEMM_EINVAL_PTR, "dtypes, sizes or X is NULL");
    for (int64_t i = 0; i < count; ++i) {
        if (!float_type(dtypes[i]))
            return fail(SGEMM_EINVAL_TYPE, "dtypes[%lld]=%d", (long long)i, dtypes[i]);
        if (sizes[i] < 0 || sizes[i] > (int64_t)1 << 40)
            return fail(SGEMM_EINVAL_DIM, "sizes[%lld]=%lld: must be 0 .. 2^40", (long long)i,
                        (long long)sizes[i]);
        const uintptr_t size = (uintptr_t)dtype_size(dtypes[i]);
        if (sizes[i] > 0 && (X[i] == nullptr || !aligned(X[i], size) ||
                             (Y != nullptr && (Y[i] == nullptr || !aligned(Y[i], size)))))
            return fail(SGEMM_EINVAL_PTR, "tensor %lld or its result is NULL or not aligned",
                        (long long)i);
    }
    if (Y != nullptr && !(max_norm >= 0.f && eps >= 0.f))
        return fail(SGEMM_EINVAL_DIM, "max_norm=%g, eps=%g: both must be at least 0", max_norm, eps);
    if (!aligned(norm, 4)) return fail(SGEMM_EINVAL_PTR, "norm is not 4-byte aligned");
    if (Y != nullptr) {
        bool overlap;
        try {
            overlap = results_overlap(count, dtypes, sizes, X, Y);
        } catch (const std::exception &) {
            return fail(SGEMM_EINVAL_DIM, "no host memory for a list of %lld tensors",
                        (long long)count);
        }
        if (overlap)
            return fail(SGEMM_EINVAL_PTR, "a result overlaps another one or a tensor of the list "
                        "other than its own");
    }
    if (Y == nullptr && norm == nullptr) return SGEMM_OK;
    CHECK(check_workspace(workspace, workspace_bytes, grad_clip_bytes(count, dtypes, sizes)));
    CHECK(require_device());
    return launched(launch_grad_clip(count, dtypes, sizes, X, Y, max_norm, eps, norm,
                                     static_cast<double *>(workspace), s));
}

}  // namespace
}  // namespace sgemm

extern "C" {

int sgemm_gated_linear(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                       const float *x_scale, const void *Wg, int64_t ldwg, const float *gate_scale,
                       const void *Wu, int64_t ldwu, const float *up_scale, int transW,
                       const void *bias_gate, const void *bias_up, int activation, int out_dtype,
                       void *H, int64_t ldh, void *preact_gate, int64_t ldpg, void *preact_up,
                       int64_t ldpu, void *workspace, uint64_t workspace_bytes, void *stream) {
    return sgemm::gated_linear(dtype, M, N, K, X, ldx, x_scale, Wg, ldwg, gate_scale, Wu, ldwu,
                               up_scale, transW, bias_gate, bias_up, activation, out_dtype, H, ldh,
                               preact_gate, ldpg, preact_up, ldpu, workspace, workspace_bytes,
                               static_cast<cudaStream_t>(stream));
}

uint64_t sgemm_gated_linear_workspace_size(int dtype, int64_t M, int64_t N, int64_t K,
                                           const void *X, int64_t ldx, const void *Wg, int64_t ldwg,
                                           const void *Wu, int64_t ldwu, int transW) {
    if (M <= 0 || N <= 0 || K <= 0 || dtype < SGEMM_F32 || dtype > SGEMM_E4M3) return 0;
    return sgemm::gated_bytes(dtype, M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, transW);
}

int sgemm_gated_linear_backward(int dtype, int64_t M, int64_t N, int64_t K, const void *dH,
                                int64_t lddh, const void *Zg, int64_t ldzg, const void *Zu,
                                int64_t ldzu, int activation, const void *X, int64_t ldx,
                                const void *Wg, int64_t ldwg, const void *Wu, int64_t ldwu,
                                int transW, void *dX, int64_t lddx, void *dWg, int64_t lddwg,
                                void *dWu, int64_t lddwu, void *db_gate, void *db_up,
                                void *workspace, uint64_t workspace_bytes, void *stream) {
    return sgemm::gated_linear_backward(dtype, M, N, K, dH, lddh, Zg, ldzg, Zu, ldzu, activation, X,
                                        ldx, Wg, ldwg, Wu, ldwu, transW, dX, lddx, dWg, lddwg, dWu,
                                        lddwu, db_gate, db_up, workspace, workspace_bytes,
                                        static_cast<cudaStream_t>(stream));
}

uint64_t sgemm_gated_linear_backward_workspace_size(int dtype, int64_t M, int64_t N, int64_t K,
                                                    const void *X, int64_t ldx, const void *Wg,
                                                    int64_t ldwg, const void *Wu, int64_t ldwu,
                                                    int transW) {
    if (M <= 0 || N <= 0 || K < 0 || !sgemm::float_type(dtype)) return 0;
    return sgemm::gated_backward_plan(dtype, M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, transW, true, true,
                                      true)
        .total();
}

int sgemm_add_layernorm(int dtype, int64_t rows, int64_t D, const void *X, int64_t ldx,
                        const void *residual, int64_t ldr, const void *weight, const void *bias,
                        float eps, void *S, int64_t lds, void *Y, int64_t ldy, float *q_scale,
                        float *mean, float *rstd, void *stream) {
    using namespace sgemm;
    CHECK(check_norm(dtype, rows, D));
    // (rows of no elements have a scale and statistics all the same)
    if (rows == 0 || (D == 0 && q_scale == nullptr && mean == nullptr && rstd == nullptr))
        return SGEMM_OK;
    const int size = dtype_size(dtype);
    CHECK(check_matrix("X", X, ldx, D, size, D > 0));
    CHECK(check_matrix("residual", residual, ldr, D, size, false));
    CHECK(check_matrix("S", S, lds, D, size, false));
    CHECK(check_matrix("Y", Y, ldy, D, q_scale != nullptr ? 1 : size, D > 0));
    CHECK(check_matrix("weight", weight, D > 1 ? D : 1, D, size, D > 0));
    if (!aligned(bias, (uintptr_t)size)) return fail(SGEMM_EINVAL_PTR, "bias is not aligned");
    if (!aligned(q_scale, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(SGEMM_EINVAL_PTR, "q_scale, mean or rstd is not 4-byte aligned");
    CHECK(require_device());
    return launched(launch_add_layernorm(dtype, rows, D, X, ldx, residual, ldr, weight, bias, eps, S,
                                         lds, Y, ldy, q_scale, mean, rstd,
                                         static_cast<cudaStream_t>(stream)));
}

int sgemm_add_layernorm_backward(int dtype, int64_t rows, int64_t D, const void *dY, int64_t lddy,
                                 const void *S, int64_t lds, const float *mean, const float *rstd,
                                 const void *weight, const void *dS, int64_t ldds, void *dX,
                                 int64_t lddx, void *dweight, void *dbias, void *workspace,
                                 uint64_t workspace_bytes, void *stream) {
    using namespace sgemm;
    CHECK(check_norm(dtype, rows, D));
    if (D == 0) return SGEMM_OK;
    const int size = dtype_size(dtype);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!aligned(dweight, (uintptr_t)size) || !aligned(dbias, (uintptr_t)size))
        return fail(SGEMM_EINVAL_PTR, "dweight or dbias is not aligned");
    if (rows == 0) {   // empty sums
        if (dweight == nullptr && dbias == nullptr) return SGEMM_OK;
        CHECK(require_device());
        cudaError_t e = cudaSuccess;
        for (void *d : {dweight, dbias})
            if (d != nullptr && e == cudaSuccess) e = cudaMemsetAsync(d, 0, D * size, s);
        return launched(e);
    }
    CHECK(check_matrix("dY", dY, lddy, D, size, true));
    CHECK(check_matrix("S", S, lds, D, size, true));
    CHECK(check_matrix("weight", weight, D, D, size, true));
    CHECK(check_matrix("mean", mean, 1, 1, 4, true));
    CHECK(check_matrix("rstd", rstd, 1, 1, 4, true));
    CHECK(check_matrix("dS", dS, ldds, D, size, false));
    CHECK(check_matrix("dX", dX, lddx, D, size, true));
    if (dweight != nullptr || dbias != nullptr)
        CHECK(check_workspace(workspace, workspace_bytes,
                              sgemm_add_layernorm_backward_workspace_size(dtype, rows, D)));
    CHECK(require_device());
    return launched(launch_add_layernorm_backward(dtype, rows, D, dY, lddy, S, lds, mean, rstd,
                                                  weight, dS, ldds, dX, lddx, dweight, dbias,
                                                  static_cast<float *>(workspace), s));
}

uint64_t sgemm_add_layernorm_backward_workspace_size(int dtype, int64_t rows, int64_t D) {
    if (rows <= 0 || D <= 0 || !sgemm::float_type(dtype)) return 0;
    return (uint64_t)sgemm::layernorm_backward_parts(dtype, rows, D) * 2 * (uint64_t)D *
           sizeof(float);
}

int sgemm_clip_grad_norm(int64_t count, const int *dtypes, const int64_t *sizes,
                         const void *const *X, void *const *Y, float max_norm, float eps,
                         float *norm, void *workspace, uint64_t workspace_bytes, void *stream) {
    return sgemm::clip_grad_norm(count, dtypes, sizes, X, Y, max_norm, eps, norm, workspace,
                                 workspace_bytes, static_cast<cudaStream_t>(stream));
}

uint64_t sgemm_clip_grad_norm_workspace_size(int64_t count, const int *dtypes,
                                             const int64_t *sizes) {
    if (count < 0 || (count > 0 && (dtypes == nullptr || sizes == nullptr))) return 0;
    for (int64_t i = 0; i < count; ++i)
        if (!sgemm::float_type(dtypes[i])) return 0;
    return sgemm::grad_clip_bytes(count, dtypes, sizes);
}

}  // extern "C"
