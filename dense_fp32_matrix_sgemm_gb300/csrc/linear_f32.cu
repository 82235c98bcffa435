// f32 products of the linear layer on the bf16 tensor cores, at FP32 accuracy.
//
// An f32 x is the exact sum of three bf16 values: x0 = x cut to its upper 16
// bits, x1 = bf16(x - x0) and x2 = x - x0 - x1 (24 bits of significand in
// pieces of 8), so
//   a b = a0 b0 + (a0 b1 + a1 b0) + (a1 b1 + a0 b2 + a2 b0) + dropped terms,
// the dropped ones below 2^-21 |a b| (|x1| < 2^-7 |x|, |x2| < 2^-16 |x|).  Six
// bf16 products cost what three TF32 products would, but the bf16 operands are
// half as wide, and the tensor core takes them K-major or MN-major, so no
// operand is transposed, forward or backward.
//   split3_kernel writes the three planes of both operands in the orientation
//     they are stored in (HBM-bound: 4 bytes read, 6 written an element);
//   linear_f32_kernel is linear_tc_kernel's pipeline on them: a stage is 64 of
//     K of the six tiles, and its 24 MMAs use each tile two or four times.
// The ring's slots hold one plane of both operands each, not a whole stage, and
// the MMAs go through the planes in the order a1 b1, a1 b0, a0 b1, a2 b0, a0 b2,
// a0 b0: the first ones run when two thirds of a stage have landed, and a single
// CTA gives plane 1's slot back half-way through (4096^3 in 128-wide tiles: 547
// -> 523 us).  Pairs give all three back at the end, as every commit there goes to
// both CTAs (4096^3 464 us; one a plane as it is done 482, whole stages 473).
// The tensor cores add into their accumulator with a rounding towards zero, so
// a long sum there would collect errors of one sign.  Here an accumulator
// takes one stage: the five small terms first, while it is small, then a0 b0
// (four updates at full size), and the epilogue warps add it to running sums in
// registers with ordinary fp32 adds while the other accumulators fill.
// Relative error against 64 bits, 2049 x 3071 x 1537: 8e-8 (FP32 FMAs 4.2e-7).
// 4096^3 runs at 1.84 PFLOP/s of bf16 products, what a long bf16 product runs at
// under the power limit.  128 x 128 tiles of single CTAs are bound by shared memory
// (24 MMAs read 8 KB each and the copies write 96 KB, 2250 clocks at 128 bytes a
// clock against 1536 of MMAs), so they are left to problems of few rows.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "linear_f32_kernel.cuh"

namespace sgemm {
namespace ltc {
namespace f32 {

template <int CTAS, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
linear_f32_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmY,
                  const __grid_constant__ Params<LayerEpi> p) {
    linear_f32_body<kPlain, CTAS, BN, SPLIT>({&tmA, &tmA, &tmB, &tmB, &tmY, &tmY, &tmY}, p);
}

// ------------------------------------------------------------------ split

// One operand: rows x cols of f32 as stored, its planes [3][rows][ldp] of bf16.
struct SplitJob {
    const float *X;
    __nv_bfloat16 *out;
    int64_t ld, ldp, rows;
    int cols, vec, blocks;
};
struct SplitArgs {
    SplitJob job[3];
    int chain;
};

// CTAs [0, job[0].blocks) take the first operand, the next job[1].blocks the second, the
// rest the third.  A warp
// takes pieces of 512 columns of a row, every load of a piece in flight: 16-byte
// loads of 8 columns a lane, or (rows that are not aligned) single ones of 4, which
// store 8 bytes a plane (2049 x 3071 x 1537: with 2 columns a lane the layer took
// 89 us, so 86).  From piece to piece it steps without a division.  A lane's
// loads share their sectors through L1, hence the fence (chain_begin; from L2 alone
// 2049 x 3071 x 1537 takes 107 us, 2560 x 2560 x 2600 149 for 143).
__global__ void __launch_bounds__(256) split3_kernel(const SplitArgs a) {
    chain_begin(a.chain);
    chain_fence(a.chain);
    int block = (int)blockIdx.x, which = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (which == i && block >= a.job[i].blocks) {
            block -= a.job[i].blocks;
            which = i + 1;
        }
    const SplitJob j = which == 0 ? a.job[0] : which == 1 ? a.job[1] : a.job[2];
    const int64_t warp = (int64_t)block * 8 + (threadIdx.x >> 5);
    const int64_t warps = (int64_t)j.blocks * 8;
    const int pieces = (j.cols + 511) / 512;
    const int64_t dr = warps / pieces;
    const int dc = (int)(warps - dr * pieces);
    int64_t r = warp / pieces;
    int pc = (int)(warp - r * pieces);
    const int64_t plane = j.rows * j.ldp;
    const int lane = threadIdx.x & 31;
    for (; r < j.rows; r += dr, pc += dc) {
        if (pc >= pieces) {
            pc -= pieces;
            if (++r >= j.rows) break;
        }
        const float *x = j.X + r * j.ld;
        __nv_bfloat16 *out = j.out + r * j.ldp;
        if (j.vec) {   // cols is a multiple of 8
            float4 u[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = pc * 512 + 256 * i + 8 * lane;
                if (c < j.cols) {
                    u[i][0] = *reinterpret_cast<const float4 *>(x + c);
                    u[i][1] = *(reinterpret_cast<const float4 *>(x + c) + 1);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = pc * 512 + 256 * i + 8 * lane;
                if (c >= j.cols) break;
                uint32_t p[4][3];
                split_pair(u[i][0].x, u[i][0].y, p[0]);
                split_pair(u[i][0].z, u[i][0].w, p[1]);
                split_pair(u[i][1].x, u[i][1].y, p[2]);
                split_pair(u[i][1].z, u[i][1].w, p[3]);
#pragma unroll
                for (int pl = 0; pl < 3; ++pl)
                    *reinterpret_cast<uint4 *>(out + pl * plane + c) =
                        make_uint4(p[0][pl], p[1][pl], p[2][pl], p[3][pl]);
            }
        } else {
            float u[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = pc * 512 + 128 * i + 4 * lane;
#pragma unroll
                for (int k = 0; k < 4; ++k) u[i][k] = c + k < j.cols ? x[c + k] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = pc * 512 + 128 * i + 4 * lane;
                if (c >= j.cols) break;
                uint32_t p[2][3];
                split_pair(u[i][0], u[i][1], p[0]);
                split_pair(u[i][2], u[i][3], p[1]);
#pragma unroll
                for (int pl = 0; pl < 3; ++pl)   // (the planes' rows are padded to 64)
                    *reinterpret_cast<uint2 *>(out + pl * plane + c) = make_uint2(p[0][pl], p[1][pl]);
            }
        }
    }
    chain_end(a.chain);
}

// ------------------------------------------------------------------ host side

template <int CTAS, int BN, bool SPLIT>
cudaError_t launch(const F32Planes &A, const F32Planes &B, int K, const LayerEpi &epi,
                   const Piece &piece, int chain, cudaStream_t s) {
    using S = Shape<CTAS, BN, SPLIT>;
    static PerContext<bool> configured;
    bool done = false;
    cudaError_t e;
    if (!configured.get(current_context_id(), done)) {
        e = cudaFuncSetAttribute(linear_f32_kernel<CTAS, BN, SPLIT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    Params<LayerEpi> p;
    p.epi = epi;
    const int a_rows = fill_params<CTAS, BN>(p, epi.M, epi.N, K, A.kmajor, B.kmajor, piece, chain);
    CUtensorMap tmA, tmB, tmY = {};
    p.tma = !SPLIT && stores_by_tma(epi, &tmY);
    if (!plane_map(&tmA, A.planes, A.rows, A.cols, A.kmajor ? a_rows : 64) ||
        !plane_map(&tmB, B.planes, B.rows, B.cols, B.kmajor ? S::BROWS : 64))
        return cudaErrorInvalidValue;
    Config c(ctas_of<CTAS, SPLIT>(piece), S::SMEM, SPLIT ? CTAS * piece.parts : CTAS, s);
    return cudaLaunchKernelEx(&c.cfg, linear_f32_kernel<CTAS, BN, SPLIT>, tmA, tmB, tmY, p);
}

}  // namespace f32
}  // namespace ltc

size_t f32_planes_bytes(int64_t rows, int64_t cols) {
    return ((size_t)ltc::f32::kPlanes * rows * f32_plane_ld(cols) * 2 + 255) / 256 * 256;
}

// Planes of one to three matrices, one launch; `out` at 256-byte boundaries.
cudaError_t launch_f32_split(const F32Operand *x, int count, int chain, cudaStream_t s) {
    using namespace ltc::f32;
    SplitArgs a = {};
    a.chain = chain;
    int blocks = 0;
    for (int i = 0; i < count; ++i) {
        SplitJob &j = a.job[i];
        j.X = x[i].X;
        j.out = static_cast<__nv_bfloat16 *>(x[i].planes);
        j.ld = x[i].ld;
        j.ldp = f32_plane_ld(x[i].cols);
        j.rows = x[i].rows;
        j.cols = (int)x[i].cols;
        j.vec = x[i].cols % 8 == 0 && x[i].ld % 4 == 0 &&
                reinterpret_cast<uintptr_t>(x[i].X) % 16 == 0;
        const int64_t need = (j.rows * ((j.cols + 511) / 512) + 7) / 8;
        j.blocks = (int)(need < 152 * 16 ? need : 152 * 16);
        blocks += j.blocks;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, split3_kernel, a);
}

// The tile and schedule by cost, as linear_tc's; a stage (64 of K, 24 MMAs) takes
// 1.6 to 1.8 us in pairs' 256-wide tiles, 0.86 to 0.98 in their 128-wide ones, and
// in single CTAs' 64- and 128-wide tiles 0.78 and 1.05 (those for few rows).  The
// choice against the others, us:
//   4096^3: 256-wide with the last 28 of 256 tiles in 2 parts 449 (whole 490,
//     128-wide pairs 460, single CTAs 514);
//   2049 x 3071 x 1537: 128-wide pairs 86 (256-wide 110, single CTAs 98);
//   64 x 4096 x 4096: 128-wide single CTAs in 4 parts 48 (64-wide in 2 56, pairs 57).
using ltc::f32::kCosts;

bool linear_f32_side_by_side(const ProductSize &a, const ProductSize &b) {
    ltc::Capacity cap;
    return ltc::capacity(cap) == cudaSuccess &&
           ltc::side_by_side(a, b, ltc::f32::kBk, cap, kCosts);
}

cudaError_t launch_linear_f32(const F32Planes &A, const F32Planes &B, int K, const LayerEpi &epi,
                              int chain, cudaStream_t s) {
    using namespace ltc;
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    if (chain & kChainHalf) cap = cap.half();
    const Plan plan = plan_tiles(epi.M, epi.N, (K + f32::kBk - 1) / f32::kBk, cap, kCosts);
    return run_plan(kCosts, plan, chain, [&](auto w, auto split, const Piece &p, int at) {
        constexpr TileShape t = kCosts.shape[w()];
        return f32::launch<t.ctas, t.bn, split()>(A, B, K, epi, p, at, s);
    });
}

}  // namespace sgemm
