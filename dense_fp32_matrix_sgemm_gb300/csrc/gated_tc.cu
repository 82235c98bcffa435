// The gated layer and the sum of two products on the tensor cores, 16-bit or e4m3
// operands: linear_tc_body (linear_tc_kernel.cuh) in its two other forms.
//
//   gated:  H[row, col] = act(sum_k X(row, k) Wg(col, k) + ..) (sum_k X(row, k) Wu(col, k) + ..)
//   sum:    D[row, col] = sum_k A1(row, k) B1(col, k) + sum_k A2(row, k) B2(col, k)
//
// A gated tile's BN accumulator columns are BN / 2 gates and, BN / 2 columns on, their
// factors, so one epilogue warp has both of an output and neither product goes
// through memory.  With a pair of CTAs the even one brings the gate's weights and the
// odd one the factor's: what a CTA loads, multiplies and holds is what it is in a
// plain product of 2 N features, and so are the tile costs; the results to write are
// half as many (unless both pre-activations are kept).  A single CTA brings 32 rows of
// each weight; weights stored K x N (64 features a line of the shared-memory layout)
// take 64 of each there.
// The sum is the gradient of the layer's input, dZg Wg + dZu Wu: one accumulator runs
// over both reductions, so it is rounded once and written once.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "linear_tc_kernel.cuh"

namespace sgemm {
namespace ltc {

template <int CTAS, int BN, class O, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
gated_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG,
                const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmH,
                const __grid_constant__ CUtensorMap tmZg, const __grid_constant__ CUtensorMap tmZu,
                const __grid_constant__ Params<GatedEpi> p) {
    linear_tc_body<kGated, CTAS, BN, O, SPLIT>({&tmX, &tmX, &tmG, &tmU, &tmH, &tmZg, &tmZu}, p);
}

template <int CTAS, int BN, class O, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
sum_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
              const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB2,
              const __grid_constant__ CUtensorMap tmY, const __grid_constant__ Params<LayerEpi> p) {
    linear_tc_body<kSum, CTAS, BN, O, SPLIT>({&tmA, &tmA2, &tmB, &tmB2, &tmY, &tmY, &tmY}, p);
}

template <int CTAS, int BN, class O, bool SPLIT>
cudaError_t launch_gated(int type, const TcOperand &X, const TcOperand &Wg, const TcOperand &Wu,
                         int K, const GatedEpi &epi, const Piece &piece, int chain,
                         cudaStream_t s) {
    using S = Shape<CTAS, BN, SPLIT>;
    constexpr int OUT = BN / 2;
    static PerContext<bool> configured;
    bool done = false;
    cudaError_t e;
    if (!configured.get(current_context_id(), done)) {
        e = configure(gated_tc_kernel<CTAS, BN, O, SPLIT>, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    if (OUT < 64 && !Wg.kmajor) return cudaErrorInvalidValue;
    Params<GatedEpi> p;
    p.epi = epi;
    const int a_rows = fill_params<CTAS, BN>(p, type, epi.M, 2 * epi.N, K, X.kmajor, Wg.kmajor,
                                             piece, chain);
    CUtensorMap tmX, tmG, tmU, tmH = {}, tmZg = {}, tmZu = {};
    if (!operand_map(&tmX, X, type, epi.M, K, a_rows) ||
        !operand_map(&tmG, Wg, type, epi.N, K, OUT) || !operand_map(&tmU, Wu, type, epi.N, K, OUT))
        return cudaErrorInvalidValue;
    p.tma = !SPLIT && epi.vec == 8 && out_map(&tmH, epi.H, epi.type, epi.ldh, epi.N, epi.M) &&
            (epi.Zg == nullptr || out_map(&tmZg, epi.Zg, epi.type, epi.ldg, epi.N, epi.M)) &&
            (epi.Zu == nullptr || out_map(&tmZu, epi.Zu, epi.type, epi.ldu, epi.N, epi.M));
    Config c(ctas_of<CTAS, SPLIT>(piece), S::SMEM, SPLIT ? CTAS * piece.parts : CTAS, s);
    return cudaLaunchKernelEx(&c.cfg, gated_tc_kernel<CTAS, BN, O, SPLIT>, tmX, tmG, tmU, tmH, tmZg,
                              tmZu, p);
}

template <int CTAS, int BN, class O, bool SPLIT>
cudaError_t launch_sum(int type, const TcOperand (&A)[2], const TcOperand (&B)[2], int K,
                       const LayerEpi &epi, const Piece &piece, int chain, cudaStream_t s) {
    using S = Shape<CTAS, BN, SPLIT>;
    static PerContext<bool> configured;
    bool done = false;
    cudaError_t e;
    if (!configured.get(current_context_id(), done)) {
        e = configure(sum_tc_kernel<CTAS, BN, O, SPLIT>, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    Params<LayerEpi> p;
    p.epi = epi;
    const int a_rows = fill_params<CTAS, BN>(p, type, epi.M, epi.N, K, A[0].kmajor, B[0].kmajor,
                                             piece, chain);
    p.kblocks = 2 * p.kblocks1;
    CUtensorMap tmA[2], tmB[2], tmY = {};
    for (int i = 0; i < 2; ++i)
        if (!operand_map(&tmA[i], A[i], type, epi.M, K, a_rows) ||
            !operand_map(&tmB[i], B[i], type, epi.N, K, S::BROWS))
            return cudaErrorInvalidValue;
    p.tma = !SPLIT && epi.vec == 16 && out_map(&tmY, epi.Y, epi.type, epi.ldy, epi.N, epi.M);
    Config c(ctas_of<CTAS, SPLIT>(piece), S::SMEM, SPLIT ? CTAS * piece.parts : CTAS, s);
    return cudaLaunchKernelEx(&c.cfg, sum_tc_kernel<CTAS, BN, O, SPLIT>, tmA[0], tmA[1], tmB[0],
                              tmB[1], tmY, p);
}

// Costs as linear_tc.cu's; the shapes differ by the weights' storage.
constexpr Costs<3> kByFeature = {{{2, 256}, {2, 128}, {1, 64}}, {0.27, 0.165, 0.15},
                                 {6.5, 5.5, 4.5}, {5.0, 3.0, 1.5}};
constexpr Costs<3> kByInput = {{{2, 256}, {2, 128}, {1, 128}}, {0.27, 0.165, 0.24}, {6.5, 5.5, 4.5},
                               {5.0, 3.0, 3.0}};

template <class O>
cudaError_t gated_dispatch(int type, const TcOperand &X, const TcOperand &Wg, const TcOperand &Wu,
                           int K, const GatedEpi &epi, cudaStream_t s) {
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    const int bk = kRowBytes / dtype_size(type);
    const int kblocks = (K + bk - 1) / bk;
    if (Wg.kmajor) {
        const Plan plan = plan_tiles(epi.M, 2 * epi.N, kblocks, cap, kByFeature);
        return run_plan(kByFeature, plan, 0, [&](auto w, auto split, const Piece &p, int at) {
            constexpr TileShape t = kByFeature.shape[w()];
            return launch_gated<t.ctas, t.bn, O, split()>(type, X, Wg, Wu, K, epi, p, at, s);
        });
    }
    const Plan plan = plan_tiles(epi.M, 2 * epi.N, kblocks, cap, kByInput);
    return run_plan(kByInput, plan, 0, [&](auto w, auto split, const Piece &p, int at) {
        constexpr TileShape t = kByInput.shape[w()];
        return launch_gated<t.ctas, t.bn, O, split()>(type, X, Wg, Wu, K, epi, p, at, s);
    });
}

template <class O>
cudaError_t sum_dispatch(int type, const TcOperand (&A)[2], const TcOperand (&B)[2], int K,
                         const LayerEpi &epi, int chain, cudaStream_t s) {
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    if (chain & kChainHalf) cap = cap.half();
    const int bk = kRowBytes / dtype_size(type);
    const Plan plan = plan_tiles(epi.M, epi.N, 2 * ((K + bk - 1) / bk), cap, kByFeature);
    return run_plan(kByFeature, plan, chain, [&](auto w, auto split, const Piece &p, int at) {
        constexpr TileShape t = kByFeature.shape[w()];
        return launch_sum<t.ctas, t.bn, O, split()>(type, A, B, K, epi, p, at, s);
    });
}

}  // namespace ltc

bool gated_side_by_side(int in_type, const ProductSize &sum, const ProductSize &product) {
    using namespace ltc;
    Capacity cap;
    if (capacity(cap) != cudaSuccess) return false;
    if (in_type == SGEMM_F32) return f32_three_side_by_side(sum, product, cap);
    const int bk = kRowBytes / dtype_size(in_type);
    return three_side_by_side({sum.M, sum.N, 2 * ((sum.K + bk - 1) / bk * bk)}, product, bk, cap,
                              kByFeature);
}

cudaError_t launch_gated_tc(int in_type, const TcOperand &X, const TcOperand &Wg,
                            const TcOperand &Wu, int K, const GatedEpi &epi, cudaStream_t s) {
    return epi.type == SGEMM_BF16
               ? ltc::gated_dispatch<__nv_bfloat16>(in_type, X, Wg, Wu, K, epi, s)
               : ltc::gated_dispatch<__half>(in_type, X, Wg, Wu, K, epi, s);
}

cudaError_t launch_sum_tc(int in_type, const TcOperand (&A)[2], const TcOperand (&B)[2], int K,
                          const LayerEpi &epi, int chain, cudaStream_t s) {
    return epi.type == SGEMM_BF16 ? ltc::sum_dispatch<__nv_bfloat16>(in_type, A, B, K, epi, chain, s)
                                  : ltc::sum_dispatch<__half>(in_type, A, B, K, epi, chain, s);
}

}  // namespace sgemm
