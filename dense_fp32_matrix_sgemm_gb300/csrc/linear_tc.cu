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

#include "linear_tc.cuh"

namespace sgemm {
namespace ltc {

template <int CTAS, int BN, bool SPLIT>
struct Shape {
    static constexpr int BROWS = BN / CTAS;   // of B in a CTA
    static constexpr int A_TILE = BM * kRowBytes;
    static constexpr int B_TILE = BROWS * kRowBytes;
    static constexpr int KS = BN == 256 ? 1 : 2;   // kRowBytes of K in a stage
    static constexpr int SUB = A_TILE + B_TILE;
    static constexpr int STAGE = KS * SUB;
    static constexpr int STAGING = SPLIT ? 0 : kEpiWarps * kStage;   // epilogue warps' blocks
    static constexpr int STAGES = (kSmem - 1024 - 256 - STAGING) / STAGE;
    static constexpr int ACCS = SPLIT ? 1 : 2;
    static constexpr int TMEM_COLS = ACCS * BN;
    static constexpr int BARS = 2 * STAGES + 2 * ACCS + 1;
    static constexpr int SMEM = STAGES * STAGE + STAGING + 1024 + 256;
    static_assert(TMEM_COLS >= 32 && TMEM_COLS <= 512, "tensor memory");
    static_assert(BARS * 8 + 8 <= 256, "barrier area");
    static_assert(!SPLIT || BM * BN * 4 <= STAGES * STAGE, "a part of a tile fits the ring");
};

struct Params {
    LayerEpi epi;
    int kblocks;             // K in stages
    int tiles_m, tiles_n, group_m;
    int tile0, tiles;        // this launch's tiles: tile0 .. tile0 + tiles - 1
    int chain;
    int a_kmajor, b_kmajor;
    int a_bytes;             // bytes A's boxes bring to a CTA's stage
    uint32_t idesc;
    int fp8;
    int tma;                 // Y and Z leave by TMA store, whole blocks of 32 columns
    unsigned *error;
};

// ------------------------------------------------------------------ kernel

// 32 values of this lane's row into a staging block (32 rows of 64 bytes,
// 16-byte chunk c of row r at c ^ (r >> 1 & 3): the TMA 64-byte swizzle,
// conflict-free for a quarter-warp).
template <class O>
__device__ __forceinline__ void stage_row(uint32_t block, int lane, const float (&v)[32]) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     :: "r"(block + (uint32_t)lane * 64u +
                            ((uint32_t)(c ^ ((lane >> 1) & 3)) << 4)),
                        "r"(pack2<O>(v[8 * c], v[8 * c + 1])),
                        "r"(pack2<O>(v[8 * c + 2], v[8 * c + 3])),
                        "r"(pack2<O>(v[8 * c + 4], v[8 * c + 5])),
                        "r"(pack2<O>(v[8 * c + 6], v[8 * c + 7])) : "memory");
}

// Finishes COLS columns of the 32 tile rows of TMEM lane quarter q, a row a
// lane, 32 columns at a time: the epilogue runs on the accumulators in
// registers, Y and Z leave by TMA as whole 64-byte row pieces.  What TMA cannot
// store (rows that are not 16-byte aligned, the last block of a width that is
// not a multiple of 32) passes through the staging block in fp32 and is
// finished with a column a lane.  The loop is kept rolled: a problem of one
// tile a CTA runs this code once, and fetching it cold costs more than running
// it.
template <int COLS, class O>
__device__ __forceinline__ void finish_rows(const Params &p, const void *tmY, const void *tmZ,
                                            uint32_t acc, int q, int lane, int m0, int n0,
                                            uint32_t stage) {
    const LayerEpi &e = p.epi;
    const int row0 = m0 + 32 * q;
    if (row0 >= e.M) return;
    const int row = row0 + lane;
    const bool in = row < e.M;
    const uint32_t lane_base = acc + ((uint32_t)(32 * q) << 16);
    const float sx = e.sx != nullptr && in ? e.sx[row] : 1.f;
#pragma unroll 1
    for (int c = 0; c < COLS / 32 && n0 + 32 * c < e.N; ++c) {
        const int col = n0 + 32 * c;
        const bool fast = p.tma && col + 32 <= e.N;
        uint32_t res[2][8];
        if (fast && e.R != nullptr && in) {
            const O *r = static_cast<const O *>(e.R) + row * e.ldr + col;
            load_32b(r, res[0]);
            load_32b(r + 16, res[1]);
        }
        if (lane == 0) tc::bulk_wait_group_read<0>();   // the staging block is free
        float v[32];
        __syncwarp();   // the load is warp-collective
        tc::tmem_ld_32(lane_base + (uint32_t)(32 * c), v);
        if (!fast) {
            const int rows = min(32, e.M - row0);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                tc::st_shared_v4(stage + (uint32_t)lane * 128u + ((uint32_t)(j ^ (lane & 7)) << 4),
                                 v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            __syncwarp();
            finish_staged<O, 8>(e, stage, lane, row0, rows, col + lane);
            continue;   // (the next block's __syncwarp keeps it from overwriting this one)
        }
        if (e.sx != nullptr) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 sw = *reinterpret_cast<const float4 *>(e.sw + col + j);
                v[j] *= sx * sw.x;
                v[j + 1] *= sx * sw.y;
                v[j + 2] *= sx * sw.z;
                v[j + 3] *= sx * sw.w;
            }
        }
        if (e.bias != nullptr) {
            const O *b = static_cast<const O *>(e.bias) + col;
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                const uint4 u = *reinterpret_cast<const uint4 *>(b + j);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2<O>(w[i]);
                    v[j + 2 * i] += f.x;
                    v[j + 2 * i + 1] += f.y;
                }
            }
        }
        if (e.Z != nullptr) stage_row<O>(stage + 2048u, lane, v);
        activate_all<O>(v, e.act);
        if (e.R != nullptr && in) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 f = unpack2<O>(res[i][j]);
                    v[16 * i + 2 * j] += f.x;
                    v[16 * i + 2 * j + 1] += f.y;
                }
        }
        stage_row<O>(stage, lane, v);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store(tmY, stage, col, row0);
            if (e.Z != nullptr) tma_store(tmZ, stage + 2048u, col, row0);
            tc::bulk_commit_group();
        }
    }
}

template <int CTAS, int BN, class O, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ,
                 const __grid_constant__ Params p) {
    using S = Shape<CTAS, BN, SPLIT>;
    constexpr int STAGES = S::STAGES, ACCS = S::ACCS;
    constexpr bool CLUSTER = CTAS == 2 || SPLIT;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = tc::smem_u32_generic(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw_addr & 1023)) & 1023);
    const uint32_t ring = tc::smem_u32_generic(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * S::STAGE + S::STAGING);
    const uint32_t full0 = tc::smem_u32_generic(bars);
    const uint32_t empty0 = full0 + 8 * STAGES;
    const uint32_t accf0 = empty0 + 8 * STAGES;   // accumulator b holds a finished tile
    const uint32_t acce0 = accf0 + 8 * ACCS;      // accumulator b has been drained
    const uint32_t done_bar = acce0 + 8 * ACCS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + S::BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    // (broadcast: the compiler then knows that a warp takes one role as a whole)
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = CLUSTER ? (int)cluster_rank() : 0;
    const int half = CTAS == 2 ? rank & 1 : 0;      // this CTA's half of the pair's tile
    const int leader = CTAS == 2 ? rank & ~1 : rank;
    const uint16_t mask = (uint16_t)(3u << leader);
    // this CTA's tiles first, first + stride, ... and its K blocks of each
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
        for (int s = 0; s < STAGES; ++s) {
            tc::mbar_init(full0 + 8 * s, 1);
            tc::mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < ACCS; ++b) {
            tc::mbar_init(accf0 + 8 * b, 1);
            tc::mbar_init(acce0 + 8 * b, CTAS * kEpiWarps);
        }
        tc::mbar_init(done_bar, 1);
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    // a pair's CTAs use one another's barriers: its barrier is passed while
    // tensor memory is allocated
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
    if (warp == 2 && ntiles > 0 && tc::elect_one()) {
        // the weights of the first stages into L2 while earlier work ends (L2 is where
        // that work's writes go, so nothing stale is read): a block of norm, 4096 ->
        // 8192 and back of 64 rows 39.2 -> 38.4 us in bf16, 28.8 -> 27.8 in 8 bits
        int tm, tn;
        raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first, tm, tn);
        const int n0 = tn * BN + half * S::BROWS, bk = p.fp8 ? 128 : 64;
        for (int kb = kb0; kb < min(kb1, kb0 + S::KS * STAGES); ++kb) {
            if (p.b_kmajor) {
                tma_prefetch(&tmB, kb * bk, n0);
            } else {
#pragma unroll
                for (int c = 0; c < S::BROWS / 64; ++c) tma_prefetch(&tmB, n0 + 64 * c, kb * bk);
            }
        }
    }
    __syncwarp();
    chain_begin(p.chain);   // nothing below reads or writes global memory before earlier work has finished

    if (warp == 0) {
        if (tc::elect_one()) {
            // ---------------- TMA producer: this CTA's rows of A and B
            const int bk = p.fp8 ? 128 : 64;
            const uint32_t tx = (uint32_t)(CTAS * (p.a_bytes + S::B_TILE));
            const uint32_t fulls = CTAS == 2 ? cluster_addr(full0, leader) : full0;
            tc::Ring<STAGES> r;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                int tm, tn;
                raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first + i * stride, tm, tn);
                const int m0 = (tm * CTAS + half) * BM, n0 = tn * BN + half * S::BROWS;
                for (int kb = kb0; kb < kb1; kb += S::KS) {
                    if (r.used == STAGES && !tc::wait(empty0 + 8 * r.s, r.parity ^ 1, abort_flag)) {
                        stop = true;
                        break;
                    }
                    const uint32_t fb = fulls + 8 * r.s;
                    const int subs = min(S::KS, kb1 - kb);
                    if (half == 0) tc::mbar_arrive_expect_tx(full0 + 8 * r.s, tx * subs);
#pragma unroll
                    for (int j = 0; j < S::KS; ++j) {
                        if (j >= subs) break;
                        const uint32_t st = ring + r.s * S::STAGE + j * S::SUB;
                        const int k0 = (kb + j) * bk;
                        if (p.a_kmajor) {
                            tma_load<CTAS>(st, &tmA, fb, k0, m0);
                        } else {
#pragma unroll
                            for (int c = 0; c < BM / 64; ++c)
                                tma_load<CTAS>(st + c * kBox, &tmA, fb, m0 + 64 * c, k0);
                        }
                        if (p.b_kmajor) {
                            tma_load<CTAS>(st + S::A_TILE, &tmB, fb, k0, n0);
                        } else {
#pragma unroll
                            for (int c = 0; c < S::BROWS / 64; ++c)
                                tma_load<CTAS>(st + S::A_TILE + c * kBox, &tmB, fb, n0 + 64 * c, k0);
                        }
                    }
                    r.next();
                }
            }
            // the copies of both CTAs, before the pair leaves
            if (half == 0 && *abort_flag) tc::drain_ring(r, full0);
        }
    } else if (warp == 1) {
        if (half == 0 && tc::elect_one()) {
            // ---------------- MMA issuer, for the whole pair
            const uint64_t astep = p.a_kmajor ? 2 : 128, bstep = p.b_kmajor ? 2 : 128;
            tc::Ring<STAGES> r;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                const int b = i % ACCS, u = i / ACCS;
                if (i >= ACCS && !tc::wait(acce0 + 8 * b, (u - 1) & 1, abort_flag)) break;
                tc::fence_after_sync();
                const uint32_t acc = tmem + (uint32_t)(b * BN);
                for (int kb = 0; kb < nk; kb += S::KS) {
                    if (!tc::wait(full0 + 8 * r.s, r.parity, abort_flag)) {
                        stop = true;
                        break;
                    }
                    tc::fence_after_sync();
#pragma unroll
                    for (int j = 0; j < S::KS; ++j) {
                        if (kb + j >= nk) break;
                        const uint32_t st = ring + r.s * S::STAGE + j * S::SUB;
                        const uint64_t ad = p.a_kmajor ? tc::kmajor_desc<128>(st) : mnmajor_desc(st);
                        const uint64_t bd = p.b_kmajor ? tc::kmajor_desc<128>(st + S::A_TILE)
                                                       : mnmajor_desc(st + S::A_TILE);
                        if (p.fp8) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma<CTAS, true>(acc, ad + kk * astep, bd + kk * bstep, p.idesc,
                                                (kb | j | kk) ? 1u : 0u);
                        } else {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma<CTAS, false>(acc, ad + kk * astep, bd + kk * bstep, p.idesc,
                                                 (kb | j | kk) ? 1u : 0u);
                        }
                    }
                    commit<CTAS>(empty0 + 8 * r.s, mask);
                    if (kb + S::KS >= nk) commit<CTAS>(accf0 + 8 * b, mask);
                    r.next();
                }
            }
            commit<CTAS>(done_bar, mask);   // tracks every MMA issued above, also on abort
        }
    } else {
        // ---------------- epilogue: this CTA's rows
        if (p.epi.bias != nullptr || p.epi.R != nullptr || p.epi.sx != nullptr)
            chain_fence(p.chain);   // they are read through L1
        const int q = warp & 3, side = (warp - 2) >> 2;
        const uint32_t stage = ring + STAGES * S::STAGE + (uint32_t)((warp - 2) * kStage);
        for (int i = 0; i < ntiles; ++i) {
            const int b = i % ACCS, u = i / ACCS;
            int tm, tn;
            raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first + i * stride, tm, tn);
            const int m0 = (tm * CTAS + half) * BM, n0 = tn * BN + side * (BN / 2);
            prefetch_residual<O>(p.epi, m0 + 32 * q + lane, n0, BN / 2);
            const bool ok = tc::wait(accf0 + 8 * b, u & 1, abort_flag);
            __syncwarp();
            // one warp-uniform decision: the TMEM loads are warp-collective
            if (!__all_sync(0xffffffffu, ok && !*abort_flag)) break;
            tc::fence_after_sync();
            const uint32_t acc = tmem + (uint32_t)(b * BN + side * (BN / 2));
            if constexpr (SPLIT) {
                // the sums to this CTA's shared memory, over the ring: every
                // MMA has read its operands.  Row r, 16-byte chunk c at
                // c ^ (r & 7) of its BN * 4 bytes.
                if (m0 + 32 * q < p.epi.M) {
                    const int r = 32 * q + lane;
#pragma unroll 1
                    for (int c = 0; c < BN / 64; ++c) {
                        float v[32];
                        __syncwarp();
                        tc::tmem_ld_32(acc + ((uint32_t)(32 * q) << 16) + (uint32_t)(32 * c), v);
                        const int c0 = side * (BN / 8) + 8 * c;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            tc::st_shared_v4(ring + (uint32_t)(r * BN * 4) +
                                                 ((uint32_t)((c0 + j) ^ (r & 7)) << 4),
                                             v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                }
            } else {
                finish_rows<BN / 2, O>(p, &tmY, &tmZ, acc, q, lane, m0, n0, stage);
            }
            tc::fence_before_sync();   // the TMEM loads above precede the release
            __syncwarp();
            if (lane == 0) {
                if constexpr (CTAS == 2)
                    arrive_cluster(cluster_addr(acce0 + 8 * b, leader));
                else
                    tc::mbar_arrive(acce0 + 8 * b);
            }
        }
        if (!SPLIT && lane == 0) tc::bulk_wait_group_read<0>();   // the stores have left
    }
    __syncwarp();

    tc::fence_before_sync();
    __syncthreads();
    if constexpr (SPLIT) {
        // Every CTA of the cluster passes the barriers, an aborted one too (its
        // share of the tile is then not valid, and the status word says so).
        // This CTA's rows are held by the CTAs of its half of every pair.
        cluster_sync();
        int tm, tn;
        raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first, tm, tn);
        const int m0 = (tm * CTAS + half) * BM;
        const int rows = min(BM, p.epi.M - m0);
        const int n0 = tn * BN;
        if (parts == 2) join_parts<2, CTAS, BN, O>(p.epi, ring, part, half, m0, n0, rows);
        if (parts == 4) join_parts<4, CTAS, BN, O>(p.epi, ring, part, half, m0, n0, rows);
        if (parts == 8) join_parts<8, CTAS, BN, O>(p.epi, ring, part, half, m0, n0, rows);
    }
    if (*abort_flag && threadIdx.x == 0 && p.error != nullptr) atomicOr(p.error, 1u);
    if (warp == 1 && *abort_flag) {
        // every MMA issued has completed before TMEM is freed (otherwise the
        // epilogue has waited for the last one)
        int local_abort = 0;
        (void)tc::mbar_wait(done_bar, 0, &local_abort);
        tc::fence_after_sync();
    }
    if constexpr (CLUSTER) cluster_sync();   // the cluster leaves together
    if (warp == 1) tmem_dealloc<CTAS>(tmem, S::TMEM_COLS);
    chain_end(p.chain);
}

// ------------------------------------------------------------------ host side

// K-major: [rows][K] with a box of 128 bytes x box_rows; MN-major: [K][rows]
// with a box of 64 x 64.
bool operand_map(CUtensorMap *map, const TcOperand &o, int type, int rows, int K, int box_rows) {
    return o.kmajor ? make_map(map, o.base, type, o.ld, K, rows, kRowBytes, box_rows,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B)
                    : make_map(map, o.base, type, o.ld, rows, K, kRowBytes, 64,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <int CTAS, int BN, class O, bool SPLIT>
cudaError_t launch(int type, const TcOperand &A, const TcOperand &B, int K, const LayerEpi &epi,
                   const Piece &piece, int chain, cudaStream_t s) {
    using S = Shape<CTAS, BN, SPLIT>;
    static PerContext<bool> configured;
    bool done = false;
    cudaError_t e;
    if (!configured.get(current_context_id(), done)) {
        e = cudaFuncSetAttribute(linear_tc_kernel<CTAS, BN, O, SPLIT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    Params p;
    p.epi = epi;
    const int bk = kRowBytes / dtype_size(type);
    p.kblocks = (K + bk - 1) / bk;
    p.tiles_m = (epi.M + CTAS * BM - 1) / (CTAS * BM);
    p.tiles_n = (epi.N + BN - 1) / BN;
    p.group_m = raster_group();
    p.a_kmajor = A.kmajor;
    p.b_kmajor = B.kmajor;
    // few rows: a box no higher than the rows (the tile's other rows are
    // whatever the stage held; they are computed and not stored)
    const int a_rows = epi.M < BM ? (epi.M + 7) / 8 * 8 : BM;
    p.a_bytes = A.kmajor ? a_rows * kRowBytes : S::A_TILE;
    p.idesc = instruction_desc(type, CTAS * BM, BN, A.kmajor, B.kmajor);
    p.fp8 = type == SGEMM_E4M3;
    p.error = device_error_word();
    CUtensorMap tmA, tmB, tmY = {}, tmZ = {};
    if (!operand_map(&tmA, A, type, epi.M, K, a_rows) ||
        !operand_map(&tmB, B, type, epi.N, K, S::BROWS))
        return cudaErrorInvalidValue;
    // Y and Z by TMA where every matrix of the epilogue is aligned (a store
    // writes whole 16-byte granules, so only whole blocks inside N are stored)
    auto out_map = [&](CUtensorMap *map, const void *base, int64_t ld) {
        return make_map(map, base, epi.type, ld, epi.N, epi.M, 64, 32, CU_TENSOR_MAP_L2_PROMOTION_NONE);
    };
    p.tma = !SPLIT && epi.vec == 16 && out_map(&tmY, epi.Y, epi.ldy) &&
            (epi.Z == nullptr || out_map(&tmZ, epi.Z, epi.ldz));
    p.chain = chain;
    p.tile0 = piece.tile0;
    p.tiles = piece.tiles;
    const long long most = piece.room < piece.tiles ? piece.room : piece.tiles;
    const long long ctas = CTAS * (SPLIT ? (long long)piece.tiles * piece.parts : most);
    Config c(ctas, S::SMEM, SPLIT ? CTAS * piece.parts : CTAS, s);
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
