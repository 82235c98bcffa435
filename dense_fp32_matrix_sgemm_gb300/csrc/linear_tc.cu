// The linear layer's product on the tensor cores: 16-bit or e4m3 operands,
// fp32 accumulation in tensor memory, the layer's epilogue on the way out.
//
//   D[row, col] = sum_k A(row, k) B(col, k)
//
// tcgen05.mma bounds it where all three sizes are large (2 M N K flops), HBM
// where one of them is small.  A CTA computes 128 x BN tiles with warps in
// three roles:
//   warp 0:         TMA producer: 128 bytes of K of A's and B's rows a stage,
//                   128-byte swizzle, a ring that runs on across tiles;
//   warp 1:         MMA issuer (M128 N=BN, 32 bytes of K an instruction);
//                   warp 1 owns tensor memory;
//   warps 2-9:      epilogue: TMEM lane quarter warp % 4, half of the columns.
// Operands may be K-major or (16-bit types) M/N-major in memory: the tensor
// core's descriptors take both, so no operand is transposed.
//   K-major:  box of 128 bytes of K x rows; 8-row groups 1024 bytes apart.
//   MN-major: boxes of 64 rows x 64 k; the 64 rows are the 128-byte line, 8
//             k make a 1024-byte group, the next 64 rows are 8192 bytes on.
// Two schedules:
//   persistent: one CTA an SM walks tiles; two accumulators (2 BN columns), so
//     a tile's epilogue overlaps the next one's MMAs;
//   split: problems with fewer tiles than SMs: the CTAs of a cluster take
//     equal parts of K of one tile, park their sums in their own shared memory
//     and finish a share of the tile each, adding the parts in rank order
//     through distributed shared memory (no workspace, one launch).
// Every wait is bounded; one that runs out flags the CTA, all roles drain and
// the library's device status word is raised.
#include <climits>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "device_utils.cuh"
#include "gemm_args.h"
#include "layer_math.cuh"
#include "layers.h"
#include "tc_utils.cuh"
#include "tma_encode.h"

namespace sgemm {
namespace ltc {

constexpr int BM = 128;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;   // producer, MMA issuer, epilogue
constexpr int kRowBytes = 128;      // of K in a stage
constexpr int kBox = 8192;          // MN-major box: 64 k x 128 bytes

template <int BN, bool SPLIT>
struct Shape {
    static constexpr int A_TILE = BM * kRowBytes;
    static constexpr int B_TILE = BN * kRowBytes;
    static constexpr int STAGE = A_TILE + B_TILE;
    static constexpr int STAGES = 224 * 1024 / STAGE;
    static constexpr int ACCS = SPLIT ? 1 : 2;
    static constexpr int TMEM_COLS = ACCS * BN;
    static constexpr int BARS = 2 * STAGES + 2 * ACCS + 1;
    static constexpr int SMEM = STAGES * STAGE + 1024 + 256;
    static_assert(TMEM_COLS >= 32 && TMEM_COLS <= 512, "tensor memory");
    static_assert(BARS * 8 + 8 <= 256, "barrier area");
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
    static_assert(BM * BN * 4 <= STAGES * STAGE, "the split's partial tile fits the ring");
};

struct Params {
    LayerEpi epi;
    int kblocks;             // K in stages
    int tiles_m, tiles_n, group_m;
    int a_kmajor, b_kmajor;
    int a_bytes;             // bytes A's boxes bring to a stage
    uint32_t idesc;
    int fp8;
    unsigned *error;
};

// True in one lane of a converged warp.  The producer's and the MMA issuer's
// loops run in such a lane: elect.sync tells the compiler that a single thread
// is active, so descriptors and coordinates stay in uniform registers.  In the
// same loops under "lane == 0" an MMA took about 226 clocks to issue, against
// the 128 that it runs (4096 x 8192 x 4096: 224 us, 160 elected).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Bounded wait that polls before it reads the clock or the abort word: a
// stage is handed over every 512 clocks, and those two reads in front of each
// poll alone held the pair kernel at 157 us where this takes 140.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    return tc::mbar_wait(bar, parity, abort);
}

// Position in a ring of N stages: the stage, the parity of its current round,
// and how many stages have been used so far (up to N).
template <int N>
struct Ring {
    int s = 0, parity = 0, used = 0;
    __device__ __forceinline__ void next() {
        if (used < N) ++used;
        if (++s == N) {
            s = 0;
            parity ^= 1;
        }
    }
};

// Waits (bounded) until the latest fill of every used stage has landed: a CTA
// that gave up does not leave with copies in flight.
template <int N>
__device__ __forceinline__ void drain_ring(const Ring<N> &r, uint32_t full0) {
    for (int s = 0; s < r.used; ++s) {
        const int parity = s < r.s ? r.parity : r.parity ^ 1;
        const long long t0 = clock64();
        while (!tc::mbar_try_wait(full0 + 8 * s, parity) &&
               clock64() - t0 < tc::kWaitLimitCycles) {
        }
    }
}

// 2-D tiled load of the box at (c0, c1); c0 (innermost) a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void *tmap, uint32_t bar, int c0,
                                            int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

// Descriptor of an MN-major operand tile: 64-row chunks kBox bytes apart
// (leading offset), groups of 8 k 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(kBox >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;   // 128-byte swizzle
    return d;
}

__device__ __forceinline__ void mma_f16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ void mma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ void raster(const Params &p, int t, int &tm, int &tn) {
    const int group = p.group_m * p.tiles_n;
    const int g = t / group;
    const int first = g * p.group_m;
    const int rows = min(p.tiles_m - first, p.group_m);
    const int r = t - g * group;
    tm = first + r % rows;
    tn = r / rows;
}

// Finishes COLS columns of the 32 tile rows of TMEM lane quarter q, a row a
// lane: the accumulators stay in registers from tensor memory to the store.
// Global accesses are 32 bytes a lane, whole sectors of one row each, so they
// need no exchange between lanes.  (Turning the tile through shared memory
// first, for accesses along a row, took 71 us of the 4096 x 8192 outputs of a
// plain product, and 199 with GELU and stored z, and 11 and 22 this way.)
template <int COLS, class O>
__device__ __forceinline__ void finish_rows(const LayerEpi &e, uint32_t acc, int q, int lane,
                                            int m0, int n0) {
    const int row0 = m0 + 32 * q;
    if (row0 >= e.M) return;
    const int row = row0 + lane;
    const uint32_t lane_base = acc + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
    for (int c = 0; c < COLS / 32 && n0 + 32 * c < e.N; ++c) {
        const int col = n0 + 32 * c;
        float v[32];
        __syncwarp();   // the load is warp-collective
        tc::tmem_ld_32(lane_base + (uint32_t)(32 * c), v);
        if (row >= e.M) continue;
        if (e.vec == 16 && col + 32 <= e.N) {
            finish32<O>(e, row, col, v);
        } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = v[j + i];
                if (col + j < e.N) finish<O, 8>(e, row, col + j, w);
            }
        }
    }
}

template <int BN, class O, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const Params p) {
    using S = Shape<BN, SPLIT>;
    constexpr int STAGES = S::STAGES, ACCS = S::ACCS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = tc::smem_u32_generic(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw_addr & 1023)) & 1023);
    const uint32_t ring = tc::smem_u32_generic(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * S::STAGE);
    const uint32_t full0 = tc::smem_u32_generic(bars);
    const uint32_t empty0 = full0 + 8 * STAGES;
    const uint32_t accf0 = empty0 + 8 * STAGES;   // accumulator b holds a finished tile
    const uint32_t acce0 = accf0 + 8 * ACCS;      // accumulator b has been drained
    const uint32_t done_bar = acce0 + 8 * ACCS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + S::BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this CTA's tiles first, first + stride, ... and its K blocks of each
    const int total = p.tiles_m * p.tiles_n;
    int first = (int)blockIdx.x, stride = (int)gridDim.x, kb0 = 0, kb1 = p.kblocks;
    if constexpr (SPLIT) {
        const int rank = (int)cluster_rank(), size = (int)cluster_size();
        first = (int)blockIdx.x / size;
        stride = total;
        kb0 = (int)((long long)rank * p.kblocks / size);
        kb1 = (int)((long long)(rank + 1) * p.kblocks / size);
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
            tc::mbar_init(acce0 + 8 * b, kEpiWarps);
        }
        tc::mbar_init(done_bar, 1);
        *abort_flag = 0;
        tc::fence_barrier_init();
        tc::tma_prefetch_desc(&tmA);
        tc::tma_prefetch_desc(&tmB);
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_u32_generic(tmem_slot), S::TMEM_COLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    pdl_trigger();
    pdl_wait();   // nothing below touches global memory before earlier work has finished

    if (warp == 0) {
        if (elect_one()) {
            // ---------------- TMA producer
            const int bk = p.fp8 ? 128 : 64;
            const uint32_t tx = (uint32_t)(p.a_bytes + S::B_TILE);
            Ring<STAGES> r;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                int tm, tn;
                raster(p, first + i * stride, tm, tn);
                const int m0 = tm * BM, n0 = tn * BN;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (r.used == STAGES && !wait(empty0 + 8 * r.s, r.parity ^ 1, abort_flag)) {
                        stop = true;
                        break;
                    }
                    const uint32_t st = ring + r.s * S::STAGE, fb = full0 + 8 * r.s;
                    const int k0 = kb * bk;
                    tc::mbar_arrive_expect_tx(fb, tx);
                    if (p.a_kmajor) {
                        tma_load_2d(st, &tmA, fb, k0, m0);
                    } else {
#pragma unroll
                        for (int c = 0; c < BM / 64; ++c)
                            tma_load_2d(st + c * kBox, &tmA, fb, m0 + 64 * c, k0);
                    }
                    if (p.b_kmajor) {
                        tma_load_2d(st + S::A_TILE, &tmB, fb, k0, n0);
                    } else {
#pragma unroll
                        for (int c = 0; c < BN / 64; ++c)
                            tma_load_2d(st + S::A_TILE + c * kBox, &tmB, fb, n0 + 64 * c, k0);
                    }
                    r.next();
                }
            }
            if (*abort_flag) drain_ring(r, full0);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ---------------- MMA issuer
            const uint64_t astep = p.a_kmajor ? 2 : 128, bstep = p.b_kmajor ? 2 : 128;
            Ring<STAGES> r;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                const int b = i % ACCS, u = i / ACCS;
                if (i >= ACCS && !wait(acce0 + 8 * b, (u - 1) & 1, abort_flag)) break;
                tc::fence_after_sync();
                const uint32_t acc = tmem + (uint32_t)(b * BN);
                for (int kb = 0; kb < nk; ++kb) {
                    if (!wait(full0 + 8 * r.s, r.parity, abort_flag)) {
                        stop = true;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t st = ring + r.s * S::STAGE;
                    const uint64_t ad = p.a_kmajor ? tc::kmajor_desc<128>(st) : mnmajor_desc(st);
                    const uint64_t bd = p.b_kmajor ? tc::kmajor_desc<128>(st + S::A_TILE)
                                                   : mnmajor_desc(st + S::A_TILE);
                    if (p.fp8) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f8(acc, ad + kk * astep, bd + kk * bstep, p.idesc,
                                   (kb | kk) ? 1u : 0u);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16(acc, ad + kk * astep, bd + kk * bstep, p.idesc,
                                    (kb | kk) ? 1u : 0u);
                    }
                    tc::mma_commit(empty0 + 8 * r.s);
                    if (kb + 1 == nk) tc::mma_commit(accf0 + 8 * b);
                    r.next();
                }
            }
            tc::mma_commit(done_bar);   // tracks every MMA issued above, also on abort
        }
    } else {
        // ---------------- epilogue
        const int q = warp & 3, half = (warp - 2) >> 2;
        for (int i = 0; i < ntiles; ++i) {
            const int b = i % ACCS, u = i / ACCS;
            const bool ok = wait(accf0 + 8 * b, u & 1, abort_flag);
            __syncwarp();
            // one warp-uniform decision: the TMEM loads are warp-collective
            if (!__all_sync(0xffffffffu, ok && !*abort_flag)) break;
            tc::fence_after_sync();
            int tm, tn;
            raster(p, first + i * stride, tm, tn);
            const uint32_t acc = tmem + (uint32_t)(b * BN);
            if constexpr (SPLIT) {
                // the sums to this CTA's shared memory, over the ring: every
                // MMA has read its operands.  Row r, 16-byte chunk c at
                // c ^ (r & 7) of its BN * 4 bytes.
                if (tm * BM + 32 * q < p.epi.M) {
                    const int r = 32 * q + lane;
#pragma unroll 1
                    for (int c = half * (BN / 64); c < (half + 1) * (BN / 64); ++c) {
                        float v[32];
                        tc::tmem_ld_32(acc + ((uint32_t)(32 * q) << 16) + (uint32_t)(32 * c), v);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            tc::st_shared_v4(ring + (uint32_t)(r * BN * 4) +
                                                 ((uint32_t)((8 * c + j) ^ (r & 7)) << 4),
                                             v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                }
            } else {
                finish_rows<BN / 2, O>(p.epi, acc + (uint32_t)(half * (BN / 2)), q, lane, tm * BM,
                                       tn * BN + half * (BN / 2));
            }
            tc::fence_before_sync();   // the TMEM loads above precede the release
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(acce0 + 8 * b);
        }
    }
    __syncwarp();

    if constexpr (SPLIT) {
        // Every CTA of the cluster passes both barriers, an aborted one too
        // (its share of the tile is then not valid, and the status word says so).
        const int rank = (int)cluster_rank(), size = (int)cluster_size();
        __syncthreads();
        cluster_sync();
        int tm, tn;
        raster(p, first, tm, tn);
        const int rows = min(BM, p.epi.M - tm * BM);
        for (int i = rank * kThreads + (int)threadIdx.x; i < rows * (BN / 4);
             i += size * kThreads) {
            const int r = i / (BN / 4), c = i % (BN / 4);
            const int col = tn * BN + 4 * c;
            if (col >= p.epi.N) continue;
            const float4 s = cluster_sum_f4(
                ring + (uint32_t)(r * BN * 4) + ((uint32_t)(c ^ (r & 7)) << 4), (uint32_t)size);
            const float v[4] = {s.x, s.y, s.z, s.w};
            finish<O, 4>(p.epi, tm * BM + r, col, v);
        }
        cluster_sync_relaxed();   // shared memory stays until every peer has read it
    }
    tc::fence_before_sync();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0 && p.error != nullptr) atomicOr(p.error, 1u);
    if (warp == 1) {
        // every MMA issued has completed before TMEM is freed
        int local_abort = 0;
        (void)tc::mbar_wait(done_bar, 0, &local_abort);
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, S::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ CTA pairs

// 256 x 256 tiles by pairs of CTAs (cta_group::2).  Each CTA of the pair holds
// 128 rows of A and 128 of B's 256 rows a stage (32 KB) and the 128 rows of
// the result that are its own, over all 256 columns (two accumulators fill its
// tensor memory).  One MMA of the even CTA reads both halves, so a CTA takes in
// 32 KB for the 2 x 128 x 256 x 64 flops of a stage instead of the 48 KB that a
// 128 x 256 tile of its own needs: at the tensor cores' rate 64 bytes a clock
// instead of 96, which L2 can deliver.
// Barriers:
//   full (in the even CTA): both CTAs' copies complete on it; the even CTA's
//     producer expects the bytes of both;
//   empty, accumulator full (one in each CTA): completed in both by the even
//     CTA's commits;
//   accumulator empty (in the even CTA): one arrival of each of the pair's
//     sixteen epilogue warps.
// Waits are bounded as above.  A CTA whose wait runs out stops; its peer's
// waits then run out too, the even CTA waits for every copy in flight, and
// both meet at the closing cluster barrier, so neither leaves while the other
// may still write to its shared memory.
struct Pair {
    static constexpr int BN = 256;
    static constexpr int A_TILE = BM * kRowBytes;
    static constexpr int STAGE = 2 * A_TILE;
    static constexpr int STAGES = 7;
    static constexpr int BARS = 2 * STAGES + 4 + 1;
    static constexpr int SMEM = STAGES * STAGE + 1024 + 256;
    static_assert(BARS * 8 + 8 <= 256, "barrier area");
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// The shared::cluster address of `addr` (shared::cta) in the cluster's CTA 0.
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

// As tma_load_2d, into this CTA's shared memory, completing on a barrier in
// either CTA of the pair (shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void *tmap, uint32_t bar,
                                                 int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void mma_f16_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ void mma_f8_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// Arrive on the barrier at `bar` in both CTAs once every MMA issued so far by
// this thread has completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                 ".multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"((uint16_t)3) : "memory");
}

__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                 :: "r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(slot_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                 :: "r"(taddr), "r"(ncols) : "memory");
}

// p.tiles_m counts rows of 256, p.a_bytes is unused.
template <class O>
__global__ void __launch_bounds__(kThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const Params p) {
    constexpr int STAGES = Pair::STAGES, ACCS = 2, BN = Pair::BN;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = tc::smem_u32_generic(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw_addr & 1023)) & 1023);
    const uint32_t ring = tc::smem_u32_generic(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * Pair::STAGE);
    const uint32_t full0 = tc::smem_u32_generic(bars);
    const uint32_t empty0 = full0 + 8 * STAGES;
    const uint32_t accf0 = empty0 + 8 * STAGES;
    const uint32_t acce0 = accf0 + 8 * ACCS;
    const uint32_t done_bar = acce0 + 8 * ACCS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Pair::BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int total = p.tiles_m * p.tiles_n;
    const int first = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
    const int ntiles = first < total ? (total - 1 - first) / stride + 1 : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc::mbar_init(full0 + 8 * s, 1);
            tc::mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < ACCS; ++b) {
            tc::mbar_init(accf0 + 8 * b, 1);
            tc::mbar_init(acce0 + 8 * b, 2 * kEpiWarps);
        }
        tc::mbar_init(done_bar, 1);
        *abort_flag = 0;
        tc::fence_barrier_init();
        tc::tma_prefetch_desc(&tmA);
        tc::tma_prefetch_desc(&tmB);
    }
    if (warp == 1) tmem_alloc_pair(tc::smem_u32_generic(tmem_slot), ACCS * BN);
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers are initialised
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    pdl_trigger();
    pdl_wait();   // nothing below touches global memory before earlier work has finished

    if (warp == 0) {
        if (elect_one()) {
            // ---------------- TMA producer: this CTA's halves of A and B
            const int bk = p.fp8 ? 128 : 64;
            const uint32_t full_leader = leader_addr(full0);
            Ring<STAGES> r;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                int tm, tn;
                raster(p, first + i * stride, tm, tn);
                const int m0 = tm * 2 * BM + rank * BM, n0 = tn * BN + rank * (BN / 2);
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if (r.used == STAGES && !wait(empty0 + 8 * r.s, r.parity ^ 1, abort_flag)) {
                        stop = true;
                        break;
                    }
                    const uint32_t st = ring + r.s * Pair::STAGE, fb = full_leader + 8 * r.s;
                    const int k0 = kb * bk;
                    if (rank == 0) tc::mbar_arrive_expect_tx(full0 + 8 * r.s, 2 * Pair::STAGE);
                    if (p.a_kmajor) {
                        tma_load_2d_pair(st, &tmA, fb, k0, m0);
                    } else {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            tma_load_2d_pair(st + c * kBox, &tmA, fb, m0 + 64 * c, k0);
                    }
                    if (p.b_kmajor) {
                        tma_load_2d_pair(st + Pair::A_TILE, &tmB, fb, k0, n0);
                    } else {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            tma_load_2d_pair(st + Pair::A_TILE + c * kBox, &tmB, fb,
                                             n0 + 64 * c, k0);
                    }
                    r.next();
                }
            }
            // both CTAs' copies, before the pair leaves
            if (rank == 0 && *abort_flag) drain_ring(r, full0);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            // ---------------- MMA issuer, for both CTAs
            const uint64_t astep = p.a_kmajor ? 2 : 128, bstep = p.b_kmajor ? 2 : 128;
            Ring<STAGES> r;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                const int b = i % ACCS, u = i / ACCS;
                if (i >= ACCS && !wait(acce0 + 8 * b, (u - 1) & 1, abort_flag)) break;
                tc::fence_after_sync();
                const uint32_t acc = tmem + (uint32_t)(b * BN);
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if (!wait(full0 + 8 * r.s, r.parity, abort_flag)) {
                        stop = true;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t st = ring + r.s * Pair::STAGE;
                    const uint64_t ad = p.a_kmajor ? tc::kmajor_desc<128>(st) : mnmajor_desc(st);
                    const uint64_t bd = p.b_kmajor ? tc::kmajor_desc<128>(st + Pair::A_TILE)
                                                   : mnmajor_desc(st + Pair::A_TILE);
                    if (p.fp8) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f8_pair(acc, ad + kk * astep, bd + kk * bstep, p.idesc,
                                   (kb | kk) ? 1u : 0u);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16_pair(acc, ad + kk * astep, bd + kk * bstep, p.idesc,
                                    (kb | kk) ? 1u : 0u);
                    }
                    commit_pair(empty0 + 8 * r.s);
                    if (kb + 1 == p.kblocks) commit_pair(accf0 + 8 * b);
                    r.next();
                }
            }
            commit_pair(done_bar);   // tracks every MMA issued above, also on abort
        }
    } else {
        // ---------------- epilogue: this CTA's 128 rows
        const int q = warp & 3, half = (warp - 2) >> 2;
        for (int i = 0; i < ntiles; ++i) {
            const int b = i % ACCS, u = i / ACCS;
            const bool ok = wait(accf0 + 8 * b, u & 1, abort_flag);
            __syncwarp();
            if (!__all_sync(0xffffffffu, ok && !*abort_flag)) break;
            tc::fence_after_sync();
            int tm, tn;
            raster(p, first + i * stride, tm, tn);
            finish_rows<BN / 2, O>(p.epi, tmem + (uint32_t)(b * BN + half * (BN / 2)), q, lane,
                                   tm * 2 * BM + rank * BM, tn * BN + half * (BN / 2));
            tc::fence_before_sync();   // the TMEM loads above precede the release
            __syncwarp();
            if (lane == 0) arrive_cluster(leader_addr(acce0 + 8 * b));
        }
    }
    __syncwarp();

    tc::fence_before_sync();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0 && p.error != nullptr) atomicOr(p.error, 1u);
    if (warp == 1) {
        // every MMA issued has completed before TMEM is freed
        int local_abort = 0;
        (void)tc::mbar_wait(done_bar, 0, &local_abort);
        tc::fence_after_sync();
    }
    cluster_sync();   // the pair leaves together
    if (warp == 1) tmem_dealloc_pair(tmem, ACCS * BN);
}

// ------------------------------------------------------------------ host side

CUtensorMapDataType map_type(int type) {
    return type == SGEMM_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
           : type == SGEMM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                               : CU_TENSOR_MAP_DATA_TYPE_UINT8;
}

// K-major: [rows][K] with a box of 128 bytes x box_rows; MN-major: [K][rows]
// with a box of 64 x 64.
bool make_map(CUtensorMap *map, const TcOperand &o, int type, int rows, int K, int box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const int size = dtype_size(type);
    const cuuint64_t dims[2] = {(cuuint64_t)(o.kmajor ? K : rows), (cuuint64_t)(o.kmajor ? rows : K)};
    const cuuint64_t strides[1] = {(cuuint64_t)o.ld * size};
    const cuuint32_t box[2] = {(cuuint32_t)(kRowBytes / size), (cuuint32_t)(o.kmajor ? box_rows : 64)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, map_type(type), 2, const_cast<void *>(o.base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint32_t instruction_desc(int type, int bm, int bn, bool a_kmajor, bool b_kmajor) {
    const uint32_t fmt = type == SGEMM_BF16 ? 1u : 0u;   // f16 and e4m3: 0
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_kmajor ? 0u : 1u) << 15) |
           ((b_kmajor ? 0u : 1u) << 16) | ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(bm >> 4) << 24);
}

template <int BN, class O, bool SPLIT>
cudaError_t launch(int type, const TcOperand &A, const TcOperand &B, int K, const LayerEpi &epi,
                   int split, int sms, cudaStream_t s) {
    using S = Shape<BN, SPLIT>;
    static PerContext<bool> configured;
    const unsigned long long ctx = current_context_id();
    bool done = false;
    cudaError_t e;
    if (!configured.get(ctx, done)) {
        e = cudaFuncSetAttribute(linear_tc_kernel<BN, O, SPLIT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.put(current_context_id(), true);
    }
    Params p;
    p.epi = epi;
    const int bk = kRowBytes / dtype_size(type);
    p.kblocks = (K + bk - 1) / bk;
    p.tiles_m = (epi.M + BM - 1) / BM;
    p.tiles_n = (epi.N + BN - 1) / BN;
    p.group_m = raster_group();
    p.a_kmajor = A.kmajor;
    p.b_kmajor = B.kmajor;
    // few rows: a box no higher than the rows (the tile's other rows are
    // whatever the stage held; they are computed and not stored)
    const int a_rows = epi.M < BM ? (epi.M + 7) / 8 * 8 : BM;
    p.a_bytes = A.kmajor ? a_rows * kRowBytes : S::A_TILE;
    p.idesc = instruction_desc(type, BM, BN, A.kmajor, B.kmajor);
    p.fp8 = type == SGEMM_E4M3;
    p.error = device_error_word();
    CUtensorMap tmA, tmB;
    if (!make_map(&tmA, A, type, epi.M, K, a_rows) || !make_map(&tmB, B, type, epi.N, K, BN))
        return cudaErrorInvalidValue;
    const long long tiles = (long long)p.tiles_m * p.tiles_n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(SPLIT ? tiles * split : tiles < sms ? tiles : sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_tc_kernel<BN, O, SPLIT>, tmA, tmB, p);
}

// Clusters of two linear_pair_kernel CTAs that the device holds at once (an
// SM without a partner in its group of SMs holds none).
template <class O>
cudaError_t pair_capacity(int &pairs) {
    static PerContext<int> cached;
    const unsigned long long ctx = current_context_id();
    if (cached.get(ctx, pairs)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(linear_pair_kernel<O>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Pair::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Pair::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&pairs, linear_pair_kernel<O>, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    cached.put(current_context_id(), pairs);
    return cudaSuccess;
}

template <class O>
cudaError_t launch_pair(int type, const TcOperand &A, const TcOperand &B, int K,
                        const LayerEpi &epi, int pairs, cudaStream_t s) {
    Params p;
    p.epi = epi;
    const int bk = kRowBytes / dtype_size(type);
    p.kblocks = (K + bk - 1) / bk;
    p.tiles_m = (epi.M + 2 * BM - 1) / (2 * BM);
    p.tiles_n = (epi.N + Pair::BN - 1) / Pair::BN;
    p.group_m = raster_group();
    p.a_kmajor = A.kmajor;
    p.b_kmajor = B.kmajor;
    p.a_bytes = 0;
    p.idesc = instruction_desc(type, 2 * BM, Pair::BN, A.kmajor, B.kmajor);
    p.fp8 = type == SGEMM_E4M3;
    p.error = device_error_word();
    CUtensorMap tmA, tmB;
    if (!make_map(&tmA, A, type, epi.M, K, BM) || !make_map(&tmB, B, type, epi.N, K, Pair::BN / 2))
        return cudaErrorInvalidValue;
    const long long tiles = (long long)p.tiles_m * p.tiles_n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Pair::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, linear_pair_kernel<O>, tmA, tmB, p);
}

template <class O>
cudaError_t dispatch(int type, const TcOperand &A, const TcOperand &B, int K, const LayerEpi &epi,
                     cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int bk = kRowBytes / dtype_size(type);
    const int kblocks = (K + bk - 1) / bk;
    auto tiles = [&](int bn) {
        return (long long)((epi.M + BM - 1) / BM) * ((epi.N + bn - 1) / bn);
    };
    // parts of K for tiles that leave at least half the SMs idle
    auto parts = [&](int bn) {
        int n = 1;
        while (n < 8 && tiles(bn) * n * 2 <= sms && n * 4 <= kblocks) n *= 2;
        return n;
    };
    if (tiles(128) * 2 <= sms) {
        const int n64 = parts(64), n128 = parts(128);
        if (tiles(64) * n64 >= tiles(128) * n128)
            return launch<64, O, true>(type, A, B, K, epi, n64, sms, s);
        return launch<128, O, true>(type, A, B, K, epi, n128, sms, s);
    }
    // waves of one tile an SM or a pair; a pair's 256 x 256 tile is four 128 x
    // 128 ones on two SMs
    int pairs = 0;
    e = pair_capacity<O>(pairs);
    if (e != cudaSuccess) return e;
    const long long t256 = (long long)((epi.M + 255) / 256) * ((epi.N + 255) / 256);
    const double wide = 1.4 * (double)((t256 + pairs - 1) / pairs);
    const double narrow = (double)((tiles(128) + sms - 1) / sms);
    return wide <= narrow ? launch_pair<O>(type, A, B, K, epi, pairs, s)
                          : launch<128, O, false>(type, A, B, K, epi, 1, sms, s);
}

}  // namespace ltc

cudaError_t launch_linear_tc(int in_type, const TcOperand &A, const TcOperand &B, int K,
                             const LayerEpi &epi, cudaStream_t s) {
    return epi.type == SGEMM_BF16 ? ltc::dispatch<__nv_bfloat16>(in_type, A, B, K, epi, s)
                                  : ltc::dispatch<__half>(in_type, A, B, K, epi, s);
}

}  // namespace sgemm
