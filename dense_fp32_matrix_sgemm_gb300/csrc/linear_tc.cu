// The linear layer's product on the tensor cores: 16-bit or e4m3 operands,
// fp32 accumulation in tensor memory, the layer's epilogue on the way out.
//
//   D[row, col] = sum_k A(row, k) B(col, k)
//
// tcgen05.mma bounds it where all three sizes are large (2 M N K flops: pairs'
// 256 x 256 tiles take 0.27 us per 128 bytes of K, what the MMAs alone take at
// the 1.88 GHz seen under this load), the operands' way from L2 into shared
// memory where the tiles are small, HBM where few rows meet a large W.  A CTA
// has ten warps in three roles:
//   warp 0:    TMA producer: KS times 128 bytes of K of A's and B's rows a
//              stage, 128-byte swizzle, a ring that runs on across tiles;
//   warp 1:    MMA issuer (32 bytes of K an instruction); owns tensor memory;
//   warps 2-9: epilogue: TMEM lane quarter warp % 4, half of the columns.
// One thread issues each role's work, and handing a stage over costs it about
// 100 clocks for the wait, 40 to 65 for the expected bytes, 65 a copy, 60 to 105
// a commit: 330 clocks in the producer and as many in the issuer, whatever the
// stage holds.  That is hidden by the 512 clocks of the 256 x 256 tiles' MMAs, not
// by smaller tiles' 128 to 256, so their stages hold two times 128 bytes of K
// (4096 x 8192 x 4096 in 64-wide tiles 417 -> 290 us, in 256 x 128 200 -> 170).
// Operands may be K-major or (16-bit types) M/N-major in memory: the tensor
// core's descriptors take both, so no operand is transposed.
//   K-major:  box of 128 bytes of K x rows; 8-row groups 1024 bytes apart.
//   MN-major: boxes of 64 rows x 64 k; the 64 rows are the 128-byte line, 8
//             k make a 1024-byte group, the next 64 rows are 8192 bytes on.
// CTAS = 2: pairs of CTAs (cta_group::2) compute 256 x 256 tiles.  Each CTA
//   holds 128 of A's rows and 128 of B's 256 a stage (32 KB) and the 128 rows
//   of the result that are its own.  One MMA of the even CTA reads both halves,
//   so a CTA takes in 32 KB for 2 x 128 x 256 x 64 flops where a 128 x 256 tile
//   of its own takes 48 and a 128 x 128 tile 64 for the same: at the tensor
//   cores' rate 64 bytes a clock instead of 96 and 128.  (4096 x 8192 x 4096:
//   140 us.)  Pairs' 256 x 128 tiles take 96 bytes a clock, where 128 x 128 tiles
//   of single CTAs would take 128 (they were: 512 x 4096 x 4096 19.4 us, the
//   pairs' 16.8).
// CTAS = 1: 128 x 64 tiles, for problems with few rows or few tiles.
// Two schedules:
//   persistent: one CTA an SM walks tiles; two accumulators, so a tile's
//     epilogue overlaps the next one's MMAs;
//   SPLIT: problems with fewer tiles than SMs: the CTAs (or pairs) of a cluster
//     take equal parts of K of one tile, park their sums in their own shared
//     memory and finish a share of the tile each, adding the parts in K order
//     through distributed shared memory (no workspace, one launch).
// Barriers, in each CTA except where noted:
//   full (even CTA of a pair): the copies of both CTAs complete on it; the
//     even CTA's producer expects the bytes of both;
//   empty, accumulator full: completed by the issuer's commits, in both CTAs;
//   accumulator empty (even CTA): one arrival of each epilogue warp of both.
// Every wait is bounded.  A CTA whose wait runs out stops; its peer's waits
// then run out too, the even CTA waits for every copy in flight, and all CTAs
// of a cluster meet at its closing barrier, so none leaves while another may
// still write to its shared memory.  The library's device status word is
// raised.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "linear_tc_kernel.cuh"

namespace sgemm {
namespace ltc {

template <int CTAS, int BN, class O, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ,
                 const __grid_constant__ Params<LayerEpi> p) {
    linear_tc_body<kPlain, CTAS, BN, O, SPLIT>({&tmA, &tmA, &tmB, &tmB, &tmY, &tmZ, &tmZ}, p);
}

// ------------------------------------------------------------------ host side

template <int CTAS, int BN, class O, bool SPLIT>
cudaError_t launch(int type, const TcOperand &A, const TcOperand &B, int K, const LayerEpi &epi,
                   const Piece &piece, int chain, cudaStream_t s) {
    using S = Shape<CTAS, BN, SPLIT>;
    static PerContext<bool> configured;
    bool done = false;
    cudaError_t e;
    if (!configured.get(current_context_id(), done)) {
        e = configure(linear_tc_kernel<CTAS, BN, O, SPLIT>, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    Params<LayerEpi> p;
    p.epi = epi;
    const int a_rows = fill_params<CTAS, BN>(p, type, epi.M, epi.N, K, A.kmajor, B.kmajor, piece,
                                             chain);
    CUtensorMap tmA, tmB, tmY = {}, tmZ = {};
    if (!operand_map(&tmA, A, type, epi.M, K, a_rows) ||
        !operand_map(&tmB, B, type, epi.N, K, S::BROWS))
        return cudaErrorInvalidValue;
    // Y and Z by TMA where every matrix of the epilogue is aligned (a store
    // writes whole 16-byte granules, so only whole blocks inside N are stored)
    p.tma = !SPLIT && epi.vec == 16 && out_map(&tmY, epi.Y, epi.type, epi.ldy, epi.N, epi.M) &&
            (epi.Z == nullptr || out_map(&tmZ, epi.Z, epi.type, epi.ldz, epi.N, epi.M));
    Config c(ctas_of<CTAS, SPLIT>(piece), S::SMEM, SPLIT ? CTAS * piece.parts : CTAS, s);
    return cudaLaunchKernelEx(&c.cfg, linear_tc_kernel<CTAS, BN, O, SPLIT>, tmA, tmB, tmY, tmZ, p);
}

cudaError_t capacity(Capacity &cap) {
    using S = Shape<2, 256, true>;
    static PerContext<Capacity> cached;
    if (cached.get(current_context_id(), cap)) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&cap.sms, cudaDevAttrMultiProcessorCount, dev);
    auto kernel = linear_tc_kernel<2, 256, __nv_bfloat16, true>;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
        Config c(2 << i, S::SMEM, 2 << i, nullptr);
        c.attr[0] = c.attr[1];
        c.cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&cap.clusters[i], kernel, &c.cfg);
    }
    if (e != cudaSuccess) return e;
    if (cap.sms < 1 || cap.clusters[0] < 1) return cudaErrorInvalidConfiguration;
    cached.put(current_context_id(), cap);
    return cudaSuccess;
}

// The tile and schedule, by their cost in microseconds.  Measured on GB300
// (graph of 20 calls, bf16, weights out of L2): 128 bytes of K of a pair's
// 256-wide tile take 0.27 us, of its 128-wide tile 0.16 to 0.18, of a single CTA's
// 64-wide tile 0.15 to 0.17; what does not depend on K is 6.5, 5.5 and 4.5 us a
// launch; joining the parts of a split tile 1 us and, for 128 rows, 5, 3 and 1.5
// more.  The choice against the others there, in us:
//   64 x 1024 x 4096: 64-wide in 8 or 4 parts 7.5 (whole 12.4, pairs 13.4, 21.6);
//   128 x 4096 x 4096: 64-wide in 2 12.0 (whole 14.4, 128-wide in 2 14.3);
//   256 x 4096 x 4096: 64-wide 14.5 (128-wide in 2 14.7, whole 16.6);
//   512 x 4096 x 4096: 128-wide 16.8 (256-wide 23.1, in 2 19.8, 64-wide 24.2);
//   1024 x 2048 x 8192: 128-wide or 256-wide in 2 27.8 (256-wide 39.6);
//   2048^3: 256-wide 15.1 (128-wide 16.1); 1024^3: 64-wide 5.8 (6.8, 9.5);
//   4096 x 4096 x 8192: 256-wide, the last 28 of 256 tiles in 2 parts 151.9 (155.2).
constexpr Costs<3> kCosts = {{{2, 256}, {2, 128}, {1, 64}}, {0.27, 0.165, 0.15}, {6.5, 5.5, 4.5},
                             {5.0, 3.0, 1.5}};

template <class O>
cudaError_t dispatch(int type, const TcOperand &A, const TcOperand &B, int K, const LayerEpi &epi,
                     int chain, cudaStream_t s) {
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    const int bk = kRowBytes / dtype_size(type);
    if (chain & kChainHalf) cap = cap.half();
    const Plan plan = plan_tiles(epi.M, epi.N, (K + bk - 1) / bk, cap, kCosts);
    return run_plan(kCosts, plan, chain, [&](auto w, auto split, const Piece &p, int at) {
        constexpr TileShape t = kCosts.shape[w()];
        return launch<t.ctas, t.bn, O, split()>(type, A, B, K, epi, p, at, s);
    });
}

}  // namespace ltc

bool linear_tc_side_by_side(int in_type, const ProductSize &a, const ProductSize &b) {
    ltc::Capacity cap;
    return ltc::capacity(cap) == cudaSuccess &&
           ltc::side_by_side(a, b, ltc::kRowBytes / dtype_size(in_type), cap, ltc::kCosts);
}

cudaError_t launch_linear_tc(int in_type, const TcOperand &A, const TcOperand &B, int K,
                             const LayerEpi &epi, int chain, cudaStream_t s) {
    return epi.type == SGEMM_BF16 ? ltc::dispatch<__nv_bfloat16>(in_type, A, B, K, epi, chain, s)
                                  : ltc::dispatch<__half>(in_type, A, B, K, epi, chain, s);
}

}  // namespace sgemm
