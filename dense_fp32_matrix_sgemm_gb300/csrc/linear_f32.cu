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

#include "linear_tc.cuh"

namespace sgemm {
namespace ltc {
namespace f32 {

constexpr int kPlanes = 3;
constexpr int kBk = 64;   // of K in a stage

template <int CTAS, int BN, bool SPLIT>
struct Shape {
    static constexpr int BROWS = BN / CTAS;
    static constexpr int A_TILE = BM * kRowBytes;
    static constexpr int B_TILE = BROWS * kRowBytes;
    static constexpr int PLANE = A_TILE + B_TILE;   // one plane of both operands
    static constexpr int STAGING = SPLIT ? 0 : kEpiWarps * kStage;
    static constexpr int RING = (kSmem - 1024 - 256 - STAGING) / PLANE;   // planes it holds
    static constexpr int SLOTS = BN == 256 ? 2 : 4;   // accumulators, one stage's sum each
    static constexpr int TMEM_COLS = SLOTS * BN;
    static constexpr int BARS = 2 * RING + 2 * SLOTS + 1;
    static constexpr int SMEM = RING * PLANE + STAGING + 1024 + 256;
    static_assert(RING >= 2 * kPlanes, "a stage loads while another is multiplied");
    static_assert(TMEM_COLS <= 512, "tensor memory");
    static_assert(BARS * 8 + 8 <= 256, "barrier area");
    static_assert(!SPLIT || BM * BN * 4 <= RING * PLANE, "a part of a tile fits the ring");
};

struct Params {
    LayerEpi epi;
    int kblocks;
    int tiles_m, tiles_n, group_m;
    int tile0, tiles;        // this launch's tiles: tile0 .. tile0 + tiles - 1
    int chain;
    int a_kmajor, b_kmajor;
    int a_bytes;        // bytes one plane of A brings to a CTA's stage
    uint32_t idesc;
    int tma;            // Y leaves by TMA store, whole blocks of 32 columns
    unsigned *error;
};

template <int CTAS>
__device__ __forceinline__ void tma_load3(uint32_t dst, const void *tmap, uint32_t bar, int c0,
                                          int c1, int c2) {
    if constexpr (CTAS == 1)
        tc::tma_load_3d(dst, tmap, bar, c0, c1, c2);
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
            :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}

// 32 whole columns of this lane's row with bias, ReLU and residual, in
// registers, then out by TMA store through the warp's staging block (the
// 128-byte swizzle).  The other activations and a stored z take the staged path
// below: their code, unrolled over a row's registers, would be fetched longer
// than it runs.
__device__ __forceinline__ void store_row32(const LayerEpi &e, const void *tmY, uint32_t stage,
                                            int lane, int row0, int col, float (&v)[32]) {
    if (e.bias != nullptr) {
        const float4 *b = reinterpret_cast<const float4 *>(static_cast<const float *>(e.bias) + col);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 f = b[j];
            v[4 * j] += f.x;
            v[4 * j + 1] += f.y;
            v[4 * j + 2] += f.z;
            v[4 * j + 3] += f.w;
        }
    }
    if (e.act == SGEMM_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = activate<float>(v[j], SGEMM_ACT_RELU);
    }
    if (e.R != nullptr && row0 + lane < e.M) {
        const float4 *r = reinterpret_cast<const float4 *>(static_cast<const float *>(e.R) +
                                                           (row0 + lane) * e.ldr + col);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 f = r[j];
            v[4 * j] += f.x;
            v[4 * j + 1] += f.y;
            v[4 * j + 2] += f.z;
            v[4 * j + 3] += f.w;
        }
    }
    if (lane == 0) tc::bulk_wait_group_read<0>();   // the block is free
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        tc::st_shared_v4(stage + (uint32_t)lane * 128u + ((uint32_t)(j ^ (lane & 7)) << 4), v[4 * j],
                         v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store(tmY, stage, col, row0);
        tc::bulk_commit_group();
    }
}

// Roles, barriers and schedules as linear_tc_kernel; "accumulator full" and
// "empty" are per stage of K instead of per tile, counted across tiles.
template <int CTAS, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
linear_f32_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ Params p) {
    using S = Shape<CTAS, BN, SPLIT>;
    constexpr int RING = S::RING, SLOTS = S::SLOTS, COLS = BN / 2;
    constexpr bool CLUSTER = CTAS == 2 || SPLIT;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = tc::smem_u32_generic(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw_addr & 1023)) & 1023);
    const uint32_t ring = tc::smem_u32_generic(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + RING * S::PLANE + S::STAGING);
    const uint32_t full0 = tc::smem_u32_generic(bars);
    const uint32_t empty0 = full0 + 8 * RING;
    const uint32_t accf0 = empty0 + 8 * RING;   // accumulator b holds a finished stage
    const uint32_t acce0 = accf0 + 8 * SLOTS;     // accumulator b has been drained
    const uint32_t done_bar = acce0 + 8 * SLOTS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + S::BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = CLUSTER ? (int)cluster_rank() : 0;
    const int half = CTAS == 2 ? rank & 1 : 0;
    const int leader = CTAS == 2 ? rank & ~1 : rank;
    const uint16_t mask = (uint16_t)(3u << leader);
    const int total = p.tiles;
    int first = (int)blockIdx.x / CTAS, stride = (int)gridDim.x / CTAS, kb0 = 0, kb1 = p.kblocks;
    int parts = 1, part = 0;
    if constexpr (SPLIT) {
        parts = (int)cluster_size() / CTAS;
        part = rank / CTAS;
        first = (int)blockIdx.x / (CTAS * parts);
        stride = total;
        kb0 = (int)((long long)part * p.kblocks / parts);
        kb1 = (int)((long long)(part + 1) * p.kblocks / parts);
    }
    const int ntiles = first < total ? (total - 1 - first) / stride + 1 : 0;
    const int nk = kb1 - kb0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < RING; ++s) {
            tc::mbar_init(full0 + 8 * s, 1);
            tc::mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < SLOTS; ++b) {
            tc::mbar_init(accf0 + 8 * b, 1);
            tc::mbar_init(acce0 + 8 * b, CTAS * kEpiWarps);
        }
        tc::mbar_init(done_bar, 1);
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    if constexpr (CTAS == 2)
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    if (warp == 1) tmem_alloc<CTAS>(tc::smem_u32_generic(tmem_slot), S::TMEM_COLS);
    if (warp == 2 && lane == 0) {
        tc::tma_prefetch_desc(&tmA);
        tc::tma_prefetch_desc(&tmB);
    }
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (CTAS == 2) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    chain_begin(p.chain);   // nothing below touches global memory before the planes are complete

    if (warp == 0) {
        if (tc::elect_one()) {
            // ---------------- TMA producer: a stage's planes in the issuer's order
            const uint32_t tx = (uint32_t)(CTAS * (p.a_bytes + S::B_TILE));
            const uint32_t fulls = CTAS == 2 ? cluster_addr(full0, leader) : full0;
            tc::Ring<RING> r;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                int tm, tn;
                raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first + i * stride, tm, tn);
                const int m0 = (tm * CTAS + half) * BM, n0 = tn * BN + half * S::BROWS;
                for (int kb = kb0; kb < kb1 && !stop; ++kb) {
                    const int k0 = kb * kBk;
                    constexpr int order[kPlanes] = {1, 0, 2};
#pragma unroll
                    for (int j = 0; j < kPlanes; ++j) {
                        if (r.used == RING &&
                            !tc::wait(empty0 + 8 * r.s, r.parity ^ 1, abort_flag)) {
                            stop = true;
                            break;
                        }
                        const uint32_t fb = fulls + 8 * r.s;
                        const uint32_t a = ring + r.s * S::PLANE, b = a + S::A_TILE;
                        if (half == 0) tc::mbar_arrive_expect_tx(full0 + 8 * r.s, tx);
                        if (p.a_kmajor) {
                            tma_load3<CTAS>(a, &tmA, fb, k0, m0, order[j]);
                        } else {
#pragma unroll
                            for (int c = 0; c < BM / 64; ++c)
                                tma_load3<CTAS>(a + c * kBox, &tmA, fb, m0 + 64 * c, k0, order[j]);
                        }
                        if (p.b_kmajor) {
                            tma_load3<CTAS>(b, &tmB, fb, k0, n0, order[j]);
                        } else {
#pragma unroll
                            for (int c = 0; c < S::BROWS / 64; ++c)
                                tma_load3<CTAS>(b + c * kBox, &tmB, fb, n0 + 64 * c, k0, order[j]);
                        }
                        r.next();
                    }
                }
            }
            // the copies of both CTAs, before the pair leaves
            if (half == 0 && *abort_flag) tc::drain_ring(r, full0);
        }
    } else if (warp == 1) {
        if (half == 0 && tc::elect_one()) {
            // ---------------- MMA issuer, for the whole pair
            const uint64_t astep = p.a_kmajor ? 2 : 128, bstep = p.b_kmajor ? 2 : 128;
            tc::Ring<RING> r;
            tc::Ring<SLOTS> q;
            bool stop = false;
            // the next plane of the ring: its slot, once it has landed
            auto take = [&](int &slot) {
                if (!tc::wait(full0 + 8 * r.s, r.parity, abort_flag)) return false;
                slot = r.s;
                r.next();
                tc::fence_after_sync();
                return true;
            };
            for (int i = 0; i < ntiles && !stop; ++i) {
                for (int kb = 0; kb < nk; ++kb) {
                    const uint32_t acc = tmem + (uint32_t)(q.s * BN);
                    // A of one slot by B of another
                    auto term = [&](int sa, int sb, bool fresh) {
                        const uint32_t a = ring + sa * S::PLANE, b = ring + sb * S::PLANE + S::A_TILE;
                        const uint64_t ad = p.a_kmajor ? tc::kmajor_desc<128>(a) : mnmajor_desc(a);
                        const uint64_t bd = p.b_kmajor ? tc::kmajor_desc<128>(b) : mnmajor_desc(b);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma<CTAS, false>(acc, ad + kk * astep, bd + kk * bstep, p.idesc,
                                             fresh && kk == 0 ? 0u : 1u);
                    };
                    int s0, s1, s2;   // slots of the planes
                    stop = true;
                    if ((q.used == SLOTS && !tc::wait(acce0 + 8 * q.s, q.parity ^ 1, abort_flag)) ||
                        !take(s1))
                        break;
                    term(s1, s1, true);
                    if (!take(s0)) break;
                    term(s1, s0, false);
                    term(s0, s1, false);
                    if constexpr (CTAS == 1) commit<1>(empty0 + 8 * s1, mask);
                    if (!take(s2)) break;
                    term(s2, s0, false);
                    term(s0, s2, false);
                    if constexpr (CTAS == 1) commit<1>(empty0 + 8 * s2, mask);
                    term(s0, s0, false);
                    if constexpr (CTAS == 2) {
                        commit<2>(empty0 + 8 * s1, mask);
                        commit<2>(empty0 + 8 * s2, mask);
                    }
                    commit<CTAS>(empty0 + 8 * s0, mask);
                    commit<CTAS>(accf0 + 8 * q.s, mask);
                    q.next();
                    stop = false;
                }
            }
            commit<CTAS>(done_bar, mask);   // tracks every MMA issued above, also on abort
        }
    } else {
        // ---------------- epilogue: this CTA's rows, half of the columns a warp
        if (p.epi.bias != nullptr || p.epi.R != nullptr) chain_fence(p.chain);
        const int q = warp & 3, side = (warp - 2) >> 2;
        const uint32_t stage = ring + RING * S::PLANE + (uint32_t)((warp - 2) * kStage);
        tc::Ring<SLOTS> slot;
        bool stop = false;
        for (int i = 0; i < ntiles && !stop; ++i) {
            int tm, tn;
            raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first + i * stride, tm, tn);
            const int row0 = (tm * CTAS + half) * BM + 32 * q, n0 = tn * BN + side * COLS;
            prefetch_residual<float>(p.epi, row0 + lane, n0, COLS);
            float run[COLS];
#pragma unroll
            for (int j = 0; j < COLS; ++j) run[j] = 0.f;
            for (int kb = 0; kb < nk; ++kb) {
                const bool ok = tc::wait(accf0 + 8 * slot.s, slot.parity, abort_flag);
                __syncwarp();
                // one warp-uniform decision: the TMEM loads are warp-collective
                if (!__all_sync(0xffffffffu, ok && !*abort_flag)) {
                    stop = true;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t base = tmem + (uint32_t)(slot.s * BN + side * COLS) +
                                      ((uint32_t)(32 * q) << 16);
#pragma unroll
                for (int b = 0; b < COLS / 16; ++b) {
                    float v[16];
                    tc::tmem_ld_16(base + 16 * b, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) run[16 * b + j] += v[j];
                }
                tc::fence_before_sync();   // the TMEM loads above precede the release
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CTAS == 2)
                        arrive_cluster(cluster_addr(acce0 + 8 * slot.s, leader));
                    else
                        tc::mbar_arrive(acce0 + 8 * slot.s);
                }
                slot.next();
            }
            if (stop) break;
            if (row0 >= p.epi.M) continue;
            if constexpr (SPLIT) {
                // the sums to this CTA's shared memory, over the ring (every MMA
                // has read its operands): row r, 16-byte chunk c at c ^ (r & 7)
                const int r = 32 * q + lane;
#pragma unroll
                for (int j = 0; j < COLS / 4; ++j)
                    tc::st_shared_v4(ring + (uint32_t)(r * BN * 4) +
                                         ((uint32_t)((side * (COLS / 4) + j) ^ (r & 7)) << 4),
                                     run[4 * j], run[4 * j + 1], run[4 * j + 2], run[4 * j + 3]);
            } else {
                const int rows = min(32, p.epi.M - row0);
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) {
                    if (n0 + 32 * c >= p.epi.N) break;
                    if (p.tma && n0 + 32 * c + 32 <= p.epi.N) {
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = run[32 * c + j];
                        store_row32(p.epi, &tmY, stage, lane, row0, n0 + 32 * c, v);
                        continue;
                    }
                    if (lane == 0) tc::bulk_wait_group_read<0>();
                    __syncwarp();   // the block is free, the previous one has been read
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        tc::st_shared_v4(stage + (uint32_t)lane * 128u +
                                             ((uint32_t)(j ^ (lane & 7)) << 4),
                                         run[32 * c + 4 * j], run[32 * c + 4 * j + 1],
                                         run[32 * c + 4 * j + 2], run[32 * c + 4 * j + 3]);
                    __syncwarp();
                    // (a pair's running sums leave registers for eight rows)
                    finish_staged<float, BN == 256 ? 8 : 16>(p.epi, stage, lane, row0, rows,
                                                             n0 + 32 * c + lane);
                }
            }
            __syncwarp();
        }
        if (!SPLIT && lane == 0) tc::bulk_wait_group_read<0>();   // the stores have left
    }
    __syncwarp();

    tc::fence_before_sync();
    __syncthreads();
    if constexpr (SPLIT) {
        // every CTA of the cluster passes the barriers, an aborted one too
        cluster_sync();
        int tm, tn;
        raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first, tm, tn);
        const int m0 = (tm * CTAS + half) * BM;
        const int rows = min(BM, p.epi.M - m0);
        const int n0 = tn * BN;
        if (parts == 2) join_parts<2, CTAS, BN, float>(p.epi, ring, part, half, m0, n0, rows);
        if (parts == 4) join_parts<4, CTAS, BN, float>(p.epi, ring, part, half, m0, n0, rows);
        if (parts == 8) join_parts<8, CTAS, BN, float>(p.epi, ring, part, half, m0, n0, rows);
    }
    if (*abort_flag && threadIdx.x == 0 && p.error != nullptr) atomicOr(p.error, 1u);
    if (warp == 1 && *abort_flag) {
        // every MMA issued has completed before TMEM is freed (otherwise the
        // epilogue has waited for the last one)
        int local_abort = 0;
        (void)tc::mbar_wait(done_bar, 0, &local_abort);
        __syncwarp();
        tc::fence_after_sync();
    }
    if constexpr (CLUSTER) cluster_sync();   // the cluster leaves together
    if (warp == 1) tmem_dealloc<CTAS>(tmem, S::TMEM_COLS);
    chain_end(p.chain);
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
    SplitJob job[2];
    int chain;
};

// CTAs [0, job[0].blocks) take the first operand, the rest the second.  A warp
// takes pieces of 512 columns of a row, every load of a piece in flight: 16-byte
// loads of 8 columns a lane, or (rows that are not aligned) single ones of 4, which
// store 8 bytes a plane (2049 x 3071 x 1537: with 2 columns a lane the layer took
// 89 us, so 86).  From piece to piece it steps without a division.  A lane's
// loads share their sectors through L1, hence the fence (chain_begin; from L2 alone
// 2049 x 3071 x 1537 takes 107 us, 2560 x 2560 x 2600 149 for 143).
__global__ void __launch_bounds__(256) split3_kernel(const SplitArgs a) {
    chain_begin(a.chain);
    chain_fence(a.chain);
    const int which = (int)blockIdx.x < a.job[0].blocks ? 0 : 1;
    const SplitJob j = which ? a.job[1] : a.job[0];
    const int64_t warp = ((int64_t)blockIdx.x - (which ? a.job[0].blocks : 0)) * 8 +
                         (threadIdx.x >> 5);
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

// Planes as [3][rows][cols], rows f32_plane_ld(cols) apart: boxes as linear_tc's
// operands, one plane a load.  The maps end at the operand's own sizes, so the
// rows past K of an MN-major plane are zeros and not the next plane's.
bool plane_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const int64_t ld = f32_plane_ld(cols);
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, kPlanes};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(rows * ld * 2)};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

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
    Params p;
    p.epi = epi;
    p.kblocks = (K + kBk - 1) / kBk;
    p.tiles_m = (epi.M + CTAS * BM - 1) / (CTAS * BM);
    p.tiles_n = (epi.N + BN - 1) / BN;
    p.group_m = raster_group();
    p.a_kmajor = A.kmajor;
    p.b_kmajor = B.kmajor;
    const int a_rows = epi.M < BM ? (epi.M + 7) / 8 * 8 : BM;
    p.a_bytes = A.kmajor ? a_rows * kRowBytes : S::A_TILE;
    p.idesc = instruction_desc(SGEMM_BF16, CTAS * BM, BN, A.kmajor, B.kmajor);
    p.error = device_error_word();
    CUtensorMap tmA, tmB, tmY = {};
    p.tma = !SPLIT && epi.vec == 4 && epi.Z == nullptr &&
            (epi.act == SGEMM_ACT_NONE || epi.act == SGEMM_ACT_RELU) &&
            make_map(&tmY, epi.Y, SGEMM_F32, epi.ldy, epi.N, epi.M, 128, 32,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE);
    if (!plane_map(&tmA, A.planes, A.rows, A.cols, A.kmajor ? a_rows : 64) ||
        !plane_map(&tmB, B.planes, B.rows, B.cols, B.kmajor ? S::BROWS : 64))
        return cudaErrorInvalidValue;
    p.chain = chain;
    p.tile0 = piece.tile0;
    p.tiles = piece.tiles;
    const long long most = piece.room < piece.tiles ? piece.room : piece.tiles;
    const long long ctas = CTAS * (SPLIT ? (long long)piece.tiles * piece.parts : most);
    Config c(ctas, S::SMEM, SPLIT ? CTAS * piece.parts : CTAS, s);
    return cudaLaunchKernelEx(&c.cfg, linear_f32_kernel<CTAS, BN, SPLIT>, tmA, tmB, tmY, p);
}

}  // namespace f32
}  // namespace ltc

size_t f32_planes_bytes(int64_t rows, int64_t cols) {
    return ((size_t)ltc::f32::kPlanes * rows * f32_plane_ld(cols) * 2 + 255) / 256 * 256;
}

// Planes of one or two matrices, one launch; `out` at 256-byte boundaries.
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
constexpr ltc::Costs<4> kF32Costs = {{{2, 256}, {2, 128}, {1, 64}, {1, 128}}, {1.66, 0.89, 0.78, 1.05},
                                     {8.5, 8.0, 6.0, 6.0}, {5.0, 3.0, 1.5, 3.0}};

bool linear_f32_side_by_side(const ProductSize &a, const ProductSize &b) {
    ltc::Capacity cap;
    return ltc::capacity(cap) == cudaSuccess &&
           ltc::side_by_side(a, b, ltc::f32::kBk, cap, kF32Costs);
}

cudaError_t launch_linear_f32(const F32Planes &A, const F32Planes &B, int K, const LayerEpi &epi,
                              int chain, cudaStream_t s) {
    using namespace ltc;
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    if (chain & kChainHalf) cap = cap.half();
    const Plan plan = plan_tiles(epi.M, epi.N, (K + f32::kBk - 1) / f32::kBk, cap, kF32Costs);
    return run_plan(kF32Costs, plan, chain, [&](auto w, auto split, const Piece &p, int at) {
        constexpr TileShape t = kF32Costs.shape[w()];
        return f32::launch<t.ctas, t.bn, split()>(A, B, K, epi, p, at, s);
    });
}

}  // namespace sgemm
