// The gated layer and the sum of two products in f32 on the bf16 tensor cores:
// linear_f32_body (linear_f32_kernel.cuh) in its two other forms, as gated_tc.cu has them
// for the 16- and 8-bit types.  The running sums of a gate and of its factor are in the
// same lane's registers; both leave through the warp's staging block 16 outputs at a
// time, a column a lane, as unrolled activations of whole rows would be fetched longer
// than they run.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "linear_f32_kernel.cuh"

namespace sgemm {
namespace ltc {
namespace f32 {

template <int CTAS, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
gated_f32_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG,
                 const __grid_constant__ CUtensorMap tmU,
                 const __grid_constant__ Params<GatedEpi> p) {
    linear_f32_body<kGated, CTAS, BN, SPLIT>({&tmX, &tmX, &tmG, &tmU, &tmX, &tmX, &tmX}, p);
}

template <int CTAS, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
sum_f32_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
               const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB2,
               const __grid_constant__ CUtensorMap tmY,
               const __grid_constant__ Params<LayerEpi> p) {
    linear_f32_body<kSum, CTAS, BN, SPLIT>({&tmA, &tmA2, &tmB, &tmB2, &tmY, &tmY, &tmY}, p);
}

template <int CTAS, int BN, bool SPLIT>
cudaError_t launch_gated(const F32Planes &X, const F32Planes &Wg, const F32Planes &Wu, int K,
                         const GatedEpi &epi, const Piece &piece, int out, int chain,
                         cudaStream_t s) {
    using S = Shape<CTAS, BN, SPLIT>;
    static PerContext<bool> configured;
    bool done = false;
    cudaError_t e;
    if (!configured.get(current_context_id(), done)) {
        e = cudaFuncSetAttribute(gated_f32_kernel<CTAS, BN, SPLIT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    Params<GatedEpi> p;
    p.epi = epi;
    const int a_rows = fill_params<CTAS, BN>(p, epi.M, 2 * epi.N, K, X.kmajor, Wg.kmajor, piece,
                                             chain);
    p.out = out;
    p.tiles_n = (epi.N + out - 1) / out;
    p.idesc = instruction_desc(SGEMM_BF16, CTAS * BM, 2 * out, X.kmajor, Wg.kmajor);
    CUtensorMap tmX, tmG, tmU;
    if (!plane_map(&tmX, X.planes, X.rows, X.cols, X.kmajor ? a_rows : 64) ||
        !plane_map(&tmG, Wg.planes, Wg.rows, Wg.cols, Wg.kmajor ? out : 64) ||
        !plane_map(&tmU, Wu.planes, Wu.rows, Wu.cols, Wu.kmajor ? out : 64))
        return cudaErrorInvalidValue;
    Config c(ctas_of<CTAS, SPLIT>(piece), S::SMEM, SPLIT ? CTAS * piece.parts : CTAS, s);
    return cudaLaunchKernelEx(&c.cfg, gated_f32_kernel<CTAS, BN, SPLIT>, tmX, tmG, tmU, p);
}

template <int CTAS, int BN, bool SPLIT>
cudaError_t launch_sum(const F32Planes (&A)[2], const F32Planes (&B)[2], int K, const LayerEpi &epi,
                       const Piece &piece, int chain, cudaStream_t s) {
    using S = Shape<CTAS, BN, SPLIT>;
    static PerContext<bool> configured;
    bool done = false;
    cudaError_t e;
    if (!configured.get(current_context_id(), done)) {
        e = cudaFuncSetAttribute(sum_f32_kernel<CTAS, BN, SPLIT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    Params<LayerEpi> p;
    p.epi = epi;
    const int a_rows = fill_params<CTAS, BN>(p, epi.M, epi.N, K, A[0].kmajor, B[0].kmajor, piece,
                                             chain);
    p.kblocks = 2 * p.kblocks1;
    CUtensorMap tmA[2], tmB[2], tmY = {};
    p.tma = !SPLIT && stores_by_tma(epi, &tmY);
    for (int i = 0; i < 2; ++i)
        if (!plane_map(&tmA[i], A[i].planes, A[i].rows, A[i].cols, A[i].kmajor ? a_rows : 64) ||
            !plane_map(&tmB[i], B[i].planes, B[i].rows, B[i].cols, B[i].kmajor ? S::BROWS : 64))
            return cudaErrorInvalidValue;
    Config c(ctas_of<CTAS, SPLIT>(piece), S::SMEM, SPLIT ? CTAS * piece.parts : CTAS, s);
    return cudaLaunchKernelEx(&c.cfg, sum_f32_kernel<CTAS, BN, SPLIT>, tmA[0], tmA[1], tmB[0],
                              tmB[1], tmY, p);
}

// Tiles of a CTA on its own (of weights stored K x N the second: a shared-memory line is 64
// features).
constexpr Costs<2> kSingles = {{{1, 64}, {1, 128}}, {0.78, 1.05}, {6.0, 6.0}, {1.5, 3.0}};
constexpr Costs<1> kSingle = {{{1, 128}}, {1.05}, {6.0}, {3.0}};

// Pairs' tiles of 256 rows and `out` outputs, a multiple of 16 up to 128 (weights stored K x N: 64
// or 128), at costs between kCosts' widths.  The width is what makes whole rounds of the SMs:
// 1000 x 1369 x 1001 takes 44 tiles of 128 outputs on 76 pairs, 72 of 80 (42 us, 32 so).
struct Pairs {
    int out = 128;
    Plan plan;
};
Pairs plan_pairs(int M, int N, int kblocks, const Capacity &cap, bool any_out) {
    Pairs best;
    const int step = any_out ? 16 : 64;
    for (int out = step; out <= 128; out += step) {
        const Costs<1> cost = {{{2, 2 * out}}, {0.12 + 0.01203 * out}, {7.5 + 0.0078 * out},
                               {1.0 + 0.031 * out}};
        const Plan plan = plan_tiles(M, 2 * N, kblocks, cap, cost);
        if (plan.us < best.plan.us) {
            best.out = out;
            best.plan = plan;
        }
    }
    return best;
}

}  // namespace f32

bool f32_alike_side_by_side(const ProductSize &p, const Capacity &cap) {
    return alike_side_by_side(p, f32::kBk, cap, f32::kCosts, f32::kCosts);
}

}  // namespace ltc

cudaError_t launch_gated_f32(const F32Planes &X, const F32Planes &Wg, const F32Planes &Wu, int K,
                             const GatedEpi &epi, cudaStream_t s) {
    using namespace ltc;
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    const int kblocks = (K + f32::kBk - 1) / f32::kBk;
    const f32::Pairs pairs = f32::plan_pairs(epi.M, epi.N, kblocks, cap, Wg.kmajor);
    const Plan one = Wg.kmajor ? plan_tiles(epi.M, 2 * epi.N, kblocks, cap, f32::kSingles)
                               : plan_tiles(epi.M, 2 * epi.N, kblocks, cap, f32::kSingle);
    auto launch = [&](auto ctas, auto bn, auto split, const Piece &p, int out, int at) {
        return f32::launch_gated<ctas(), bn(), split()>(X, Wg, Wu, K, epi, p, out, at, s);
    };
    using std::integral_constant;
    if (one.us < pairs.plan.us) {
        const bool narrow = Wg.kmajor && one.shape == 0;
        return run_plan(f32::kSingles, one, 0, [&](auto, auto split, const Piece &p, int at) {
            const integral_constant<int, 1> single;
            return narrow ? launch(single, integral_constant<int, 64>(), split, p, 32, at)
                          : launch(single, integral_constant<int, 128>(), split, p, 64, at);
        });
    }
    return run_plan(f32::kSingle, pairs.plan, 0, [&](auto, auto split, const Piece &p, int at) {
        const integral_constant<int, 2> pair;
        return pairs.out > 64 ? launch(pair, integral_constant<int, 256>(), split, p, pairs.out, at)
                              : launch(pair, integral_constant<int, 128>(), split, p, pairs.out, at);
    });
}

cudaError_t launch_sum_f32(const F32Planes (&A)[2], const F32Planes (&B)[2], int K,
                           const LayerEpi &epi, int chain, cudaStream_t s) {
    using namespace ltc;
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    const Plan plan = plan_tiles(epi.M, epi.N, 2 * ((K + f32::kBk - 1) / f32::kBk), cap, f32::kCosts);
    return run_plan(f32::kCosts, plan, chain, [&](auto w, auto split, const Piece &p, int at) {
        constexpr TileShape t = f32::kCosts.shape[w()];
        return f32::launch_sum<t.ctas, t.bn, split()>(A, B, K, epi, p, at, s);
    });
}

}  // namespace sgemm
