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
// half as many (unless both pre-activations are kept).  A CTA on its own brings both weights'
// rows, as many of each as the launch says (weights stored K x N, 64 features a line of the
// shared-memory layout: 64).
// The sum is the gradient of the layer's input, dZg Wg + dZu Wu: one accumulator runs
// over both reductions, so it is rounded once and written once.  The weights' gradients are
// sums of one product: linear_tc.cu's, but for results of any alignment, which leave by rows
// (store_rows_any; gradients of 1000 x 1369 x 1001 bf16 38.1 -> 33.5 us).
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
                         int K, const GatedEpi &epi, const Piece &piece, int out, int chain,
                         cudaStream_t s) {
    using S = Shape<CTAS, BN, SPLIT>;
    static PerContext<bool> configured;
    bool done = false;
    cudaError_t e;
    if (!configured.get(current_context_id(), done)) {
        e = configure(gated_tc_kernel<CTAS, BN, O, SPLIT>, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    Params<GatedEpi> p;
    p.epi = epi;
    const int a_rows = fill_params<CTAS, BN>(p, type, epi.M, 2 * epi.N, K, X.kmajor, Wg.kmajor,
                                             piece, chain);
    p.out = out;
    p.tiles_n = (epi.N + out - 1) / out;
    p.a_tile = a_rows * kRowBytes;
    p.sub = p.a_tile + (3 - CTAS) * out * kRowBytes;
    // (the MMAs read 128 rows of A wherever the tile ends: the last one's stay in the ring)
    const int over = S::A_TILE > p.sub ? S::A_TILE - p.sub : 0;
    p.stages = (S::STAGES * S::STAGE - over) / (S::KS * p.sub);
    if (p.stages > kMostStages) p.stages = kMostStages;
    p.idesc = instruction_desc(type, CTAS * BM, 2 * out, X.kmajor, Wg.kmajor);
    CUtensorMap tmX, tmG, tmU, tmH = {}, tmZg = {}, tmZu = {};
    if (!operand_map(&tmX, X, type, epi.M, K, a_rows) ||
        !operand_map(&tmG, Wg, type, epi.N, K, out) || !operand_map(&tmU, Wu, type, epi.N, K, out))
        return cudaErrorInvalidValue;
    p.tma = !SPLIT && epi.vec == 8 && out_map(&tmH, epi.H, epi.type, epi.ldh, epi.N, epi.M) &&
            (epi.Zg == nullptr || out_map(&tmZg, epi.Zg, epi.type, epi.ldg, epi.N, epi.M)) &&
            (epi.Zu == nullptr || out_map(&tmZu, epi.Zu, epi.type, epi.ldu, epi.N, epi.M));
    Config c(ctas_of<CTAS, SPLIT>(piece), S::SMEM, SPLIT ? CTAS * piece.parts : CTAS, s);
    return cudaLaunchKernelEx(&c.cfg, gated_tc_kernel<CTAS, BN, O, SPLIT>, tmX, tmG, tmU, tmH, tmZg,
                              tmZu, p);
}

template <int CTAS, int BN, class O, bool SPLIT>
cudaError_t launch_sum(int type, const TcOperand (&A)[2], const TcOperand (&B)[2], int count,
                       int K, const LayerEpi &epi, const Piece &piece, int chain,
                       cudaStream_t s) {
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
    p.kblocks = count * p.kblocks1;
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

// Costs as linear_tc.cu's.
constexpr Costs<3> kSumCosts = {{{2, 256}, {2, 128}, {1, 64}}, {0.27, 0.165, 0.15},
                                {6.5, 5.5, 4.5}, {5.0, 3.0, 1.5}};
// The same beside another product: the 128-wide tiles of both share L2's way to the SMs
// (gradients of 4096 x 2816 x 1024, which took them at 0.165, 97 us; in turn 82).
constexpr Costs<3> kHalfCosts = {{{2, 256}, {2, 128}, {1, 64}}, {0.27, 0.2, 0.15}, {6.5, 5.5, 4.5},
                                 {5.0, 3.0, 1.5}};

// Pairs' tiles of 256 rows and `out` outputs (a multiple of 16 up to 128; weights stored K x N:
// 64 or 128): kSumCosts between its widths, the weights' way from HBM as in plan_single
// (here at 41 bytes a ns and SM), and tile_epilogue.
// A tile's epilogue: the eight warps take it in blocks of 32 outputs, two at a time (SiLU; 4096 x 4096
// x 128 bf16 in tiles of 128 outputs 21.7 us, of 96 24.7, of 80 28.1, of 64 25.3, of 32 39).
double tile_epilogue(int out) { return out <= 64 ? 1.45 : 2.4; }
struct Pairs {
    int out = 128;
    Plan plan;
};
Pairs plan_pairs(int M, int N, int kblocks, const Capacity &cap, bool any_out) {
    Pairs best;
    const int row_tiles = (M + 2 * BM - 1) / (2 * BM), step = any_out ? 16 : 64;
    for (int out = step; out <= 128; out += step) {
        const double l2 = out < 64 ? 0.165 : 0.06 + 0.00164 * out, hbm = 0.0031 * out / row_tiles;
        const Costs<1> cost = {{{2, 2 * out}}, {hbm > l2 ? hbm : l2},
                               {out < 64 ? 5.5 : 4.5 + 0.0156 * out}, {1.0 + 0.031 * out},
                               {tile_epilogue(out)}};
        const Plan plan = plan_tiles(M, 2 * N, kblocks, cap, cost);
        if (plan.us < best.plan.us) {
            best.out = out;
            best.plan = plan;
        }
    }
    return best;
}

// Tiles of a CTA on its own: 128 rows and `out` outputs, a multiple of 8 up to 128, in `parts`
// parts of K.  The width is what makes whole rounds of the SMs (64 x 8192 x 4096: 128 tiles of 64
// outputs leave 24 SMs idle, 256 of 32 take two rounds, 147 of 56 one).
struct Single {
    int out = 64, parts = 1;
    int64_t tiles = 0;
    double us = 1e30;
};
constexpr int kNarrow = 64, kWide = 128;   // the most outputs of either kernel

// Costs in us.  128 bytes of K take the issuing thread's three copies (0.15), the operands'
// way from L2, or, where no other row tile shares the weights, theirs from HBM at 45 bytes a ns
// and SM; the rest of a launch is 4.5, 5 % more of it all where whole tiles
// come from HBM, and joining parts 0.7 to 1.3 and 1 for 64 outputs of 128 rows.  Against the other
// choices, weights out of L2, outputs / parts:
//   64 x 8192 x 4096 bf16 56/1 24.1 (64/1 24.2, 32/1 28.4, 112/2 26.1); e4m3 56/1 15.6 (32/1 19.2)
//   64 x 11264 x 4096 bf16 80/1 31.8 (40/1 32.4, 64/1 39.9)
//   64 x 4096 x 4096 bf16 56/2 15.6 (32/1 16.4, 16/1 27.7); e4m3 56/2 10.6 (32/1 12.4)
//   64 x 1024 x 4096 bf16 32/4 8.9 (16/2 11.8, 8/1 15.4); 64 x 2048 x 1024 16/1 6.7 (32/2 7.3)
//   64 x 14336 x 4096 e4m3 48/1 23.4 (96/1 26.4)
//   256 x 4096 x 4096 bf16 pairs' 128-wide tiles 18.7 (56/1 20.6, 32/1 28.4)
//   512 x 1024 x 1024 bf16 32/1 6.7 (64/1 7.3, 64/2 8.8); 1000^3 56/1 10.3 (128/1 14.2)
Single plan_single(int M, int N, int kblocks, const Capacity &cap, bool any_out) {
    Single best;
    const int row_tiles = (M + BM - 1) / BM;
    const double rows = (M < BM ? M : BM) / (double)BM;
    for (int out = any_out ? 8 : kNarrow; out <= (any_out ? kWide : kNarrow); out += 8) {
        const int64_t tiles = (int64_t)row_tiles * ((N + out - 1) / out);
        if (tiles > 0x7fffffff) continue;
        const double l2 = 0.08 * rows + 0.0028 * out, hbm = 0.0057 * out / row_tiles;
        const double block = hbm > l2 ? hbm : l2, stage = block > 0.15 ? block : 0.15;
        for (int parts = 1; parts <= 8; parts *= 2) {
            if (parts > 1 && (tiles > cap.of(parts) || kblocks < 2 * parts)) break;
            const int64_t rounds = parts > 1 ? 1 : (tiles + cap.sms - 1) / cap.sms;
            const double product = ((kblocks + parts - 1) / parts) * stage;
            const double epilogue = 1.15 * tile_epilogue(out);   // (3000 x 4000 x 300 112/1 26.1, pairs 24.4)
            double us = product + (rounds - 1) * (product > epilogue ? product : epilogue) + 4.5;
            if (parts > 1)
                us += (parts == 2 ? 0.7 : parts == 4 ? 1.0 : 1.3) + rows * out / 64;
            else if (stage == hbm)
                us *= 1.05;
            if (us < best.us) best = {out, parts, tiles, us};
        }
    }
    return best;
}

template <class O>
cudaError_t gated_dispatch(int type, const TcOperand &X, const TcOperand &Wg, const TcOperand &Wu,
                           int K, const GatedEpi &epi, cudaStream_t s) {
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    const int bk = kRowBytes / dtype_size(type);
    const int kblocks = (K + bk - 1) / bk;
    const Pairs pairs = plan_pairs(epi.M, epi.N, kblocks, cap, Wg.kmajor);
    const Single one = plan_single(epi.M, epi.N, kblocks, cap, Wg.kmajor);
    if (one.us < pairs.plan.us) {
        const Piece p = {0, (int)one.tiles, one.parts, cap.sms};
        auto launch = [&](auto wide, auto split) {
            return launch_gated<1, 2 * (wide() ? kWide : kNarrow), O, split()>(
                type, X, Wg, Wu, K, epi, p, one.out, 0, s);
        };
        const std::true_type yes;
        const std::false_type no;
        if (one.out > kNarrow) return one.parts > 1 ? launch(yes, yes) : launch(yes, no);
        return one.parts > 1 ? launch(no, yes) : launch(no, no);
    }
    return run_plan(Costs<1>(), pairs.plan, 0, [&](auto, auto split, const Piece &p, int at) {
        return pairs.out > kNarrow
                   ? launch_gated<2, 2 * kWide, O, split()>(type, X, Wg, Wu, K, epi, p, pairs.out, at, s)
                   : launch_gated<2, 2 * kNarrow, O, split()>(type, X, Wg, Wu, K, epi, p, pairs.out, at,
                                                              s);
    });
}

template <class O>
cudaError_t sum_dispatch(int type, const TcOperand (&A)[2], const TcOperand (&B)[2], int count,
                         int K, const LayerEpi &epi, int chain, cudaStream_t s) {
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    if (chain & kChainHalf) cap = cap.half();
    const int bk = kRowBytes / dtype_size(type);
    const Plan plan = plan_tiles(epi.M, epi.N, count * ((K + bk - 1) / bk), cap,
                                 chain & kChainHalf ? kHalfCosts : kSumCosts);
    return run_plan(kSumCosts, plan, chain, [&](auto w, auto split, const Piece &p, int at) {
        constexpr TileShape t = kSumCosts.shape[w()];
        return launch_sum<t.ctas, t.bn, O, split()>(type, A, B, count, K, epi, p, at, s);
    });
}

}  // namespace ltc

bool gated_side_by_side(int in_type, const ProductSize &product) {
    using namespace ltc;
    Capacity cap;
    if (capacity(cap) != cudaSuccess) return false;
    if (in_type == SGEMM_F32) return f32_alike_side_by_side(product, cap);
    return alike_side_by_side(product, kRowBytes / dtype_size(in_type), cap, kSumCosts, kHalfCosts);
}

cudaError_t launch_gated_tc(int in_type, const TcOperand &X, const TcOperand &Wg,
                            const TcOperand &Wu, int K, const GatedEpi &epi, cudaStream_t s) {
    return epi.type == SGEMM_BF16
               ? ltc::gated_dispatch<__nv_bfloat16>(in_type, X, Wg, Wu, K, epi, s)
               : ltc::gated_dispatch<__half>(in_type, X, Wg, Wu, K, epi, s);
}

cudaError_t launch_sum_tc(int in_type, const TcOperand (&A)[2], const TcOperand (&B)[2], int count,
                          int K, const LayerEpi &epi, int chain, cudaStream_t s) {
    return epi.type == SGEMM_BF16
               ? ltc::sum_dispatch<__nv_bfloat16>(in_type, A, B, count, K, epi, chain, s)
               : ltc::sum_dispatch<__half>(in_type, A, B, count, K, epi, chain, s);
}

}  // namespace sgemm
