// The tensor-core product's kernel (described in linear_tc.cu) in its three forms:
// linear_tc.cu launches the plain one, gated_tc.cu the two others.
#pragma once

#include "linear_tc.cuh"

namespace sgemm {
namespace ltc {

constexpr int kMostStages = 12;   // of a gated tile

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

template <class E>
struct Params {
    E epi;
    int kblocks;             // K in stages
    int kblocks1;            // kSum: of the first product's K, where the second begins
    int tiles_m, tiles_n, group_m;
    int tile0, tiles;        // this launch's tiles: tile0 .. tile0 + tiles - 1
    int chain;
    int a_kmajor, b_kmajor;
    int a_bytes;             // bytes A's boxes bring to a CTA's stage
    uint32_t idesc;
    int fp8;
    int out;                 // kGated: outputs of a tile,
    int a_tile, sub, stages; //   bytes of A's rows and of 128 bytes of K in a stage, stages
    int tma;                 // Y and Z leave by TMA store, whole blocks of 32 columns
    unsigned *error;
};

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

// n of 32 values of every lane's row into rows of any alignment, through the staging block: a
// row at a time, a column a lane, or (vec >= 2: rows of whole 4-byte words, n even) two rows of
// pairs.  (Finished from fp32 a column a lane, 4096 x 4095 x 1024 took 59 us, where aligned rows
// take 39; 40 so.)
template <class O>
__device__ __forceinline__ void store_rows_any(uint32_t stage, int lane, void *base, int64_t ld,
                                               int vec, int row0, int rows, int col, int n,
                                               const float (&v)[32]) {
    __syncwarp();   // the block is free
    stage_row<O>(stage, lane, v);
    __syncwarp();
    O *const p = static_cast<O *>(base) + row0 * ld + col;
    // element (r, c): 16-byte chunk c / 8 of row r at its place of the swizzle
    if (vec >= 2 && n % 2 == 0) {
        const int c = 2 * (lane & 15), half = lane >> 4;
        O *to = p + half * ld + c;
#pragma unroll 8
        for (int r = half; r < rows; r += 2, to += 2 * ld) {
            uint32_t x;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x)
                         : "r"(stage + (uint32_t)r * 64u + ((uint32_t)((c >> 3) ^ ((r >> 1) & 3)) << 4) +
                               (uint32_t)(c & 7) * 2u) : "memory");
            if (c < n) *reinterpret_cast<uint32_t *>(to) = x;
        }
    } else {
        O *to = p + lane;
#pragma unroll 8
        for (int r = 0; r < rows; ++r, to += ld) {
            uint16_t x;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x)
                         : "r"(stage + (uint32_t)r * 64u + ((uint32_t)((lane >> 3) ^ ((r >> 1) & 3)) << 4) +
                               (uint32_t)(lane & 7) * 2u) : "memory");
            if (lane < n) *reinterpret_cast<uint16_t *>(to) = x;
        }
    }
}

// Finishes COLS columns of the 32 tile rows of TMEM lane quarter q, a row a
// lane, 32 columns at a time: the epilogue runs on the accumulators in
// registers, Y and Z leave by TMA as whole 64-byte row pieces.  What TMA cannot
// store (rows that are not 16-byte aligned, the last block of a width that is
// not a multiple of 32) passes through the staging block in fp32 and is
// finished with a column a lane (SUMS: there are no terms; by store_rows_any).  The loop is kept rolled: a problem of one
// tile a CTA runs this code once, and fetching it cold costs more than running
// it.
template <int COLS, class O, bool SUMS>
__device__ __forceinline__ void finish_rows(const Params<LayerEpi> &p, const void *tmY,
                                            const void *tmZ, uint32_t acc, int q, int lane, int m0,
                                            int n0, uint32_t stage) {
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
            if constexpr (SUMS) {
                const bool words = reinterpret_cast<uintptr_t>(e.Y) % 4 == 0 && e.ldy % 2 == 0;
                store_rows_any<O>(stage, lane, e.Y, e.ldy, words ? 2 : 1, row0, rows, col,
                                  min(32, e.N - col), v);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    tc::st_shared_v4(stage + (uint32_t)lane * 128u +
                                         ((uint32_t)(j ^ (lane & 7)) << 4),
                                     v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                __syncwarp();
                finish_staged<O, 8>(e, stage, lane, row0, rows, col + lane);
            }
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

// n (a multiple of 8) of 32 values of this lane's row as 16-byte stores.
template <class O>
__device__ __forceinline__ void store_row8s(void *base, int64_t ld, int row, int col, int n,
                                            const float (&v)[32]) {
    O *p = static_cast<O *>(base) + row * ld + col;
#pragma unroll
    for (int j = 0; j < 32; j += 8)
        if (j < n)
            *reinterpret_cast<uint4 *>(p + j) =
                make_uint4(pack2<O>(v[j], v[j + 1]), pack2<O>(v[j + 2], v[j + 3]),
                           pack2<O>(v[j + 4], v[j + 5]), pack2<O>(v[j + 6], v[j + 7]));
}

// v = v sx s[col ..] + b[col ..] for n of 32 columns, s and b of any alignment: a lane loads
// its column's terms and the warp shares them.
template <class O>
__device__ __forceinline__ void scale_and_bias_any(float (&v)[32], float sx, const float *s,
                                                   const void *b, int col, int n, int lane) {
    if (s != nullptr) {
        const float x = lane < n ? s[col + lane] : 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= sx * __shfl_sync(0xffffffffu, x, j);
    }
    if (b != nullptr) {
        const float x = lane < n ? to_f32(static_cast<const O *>(b)[col + lane]) : 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, x, j);
    }
}

// finish_rows for tiles whose accumulators hold gates and, some columns on, their factors:
// 32 outputs at a time, up to column `end`, both sums in registers.  A staging block holds
// two of the three results, so the pre-activations leave first.  (The wait for them to be
// read overlaps the next tile's MMAs.)  Fewer than 32 outputs (a tile's width is a multiple
// of 8) leave by 16-byte stores, a row a lane; what is not aligned to that passes through the
// staging block in smaller stores.
template <int BLOCKS, class O>
__device__ __forceinline__ void finish_gated_rows(const Params<GatedEpi> &p, const Maps &map,
                                                  uint32_t gate, uint32_t up, int q, int lane,
                                                  int m0, int n0, int end, uint32_t stage) {
    const GatedEpi &e = p.epi;
    const int row0 = m0 + 32 * q;
    if (row0 >= e.M) return;
    const int row = row0 + lane;
    const bool in = row < e.M, keep = e.Zg != nullptr || e.Zu != nullptr;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const float sx = e.sx != nullptr && in ? e.sx[row] : 1.f;
#pragma unroll 1
    for (int c = 0; c < BLOCKS && n0 + 32 * c < end; ++c) {
        const int col = n0 + 32 * c, n = min(32, end - col);
        if (lane == 0) tc::bulk_wait_group_read<0>();   // the staging block is free
        float v[32], u[32];
        __syncwarp();   // the loads are warp-collective
        tc::tmem_ld_32(gate + lanes + (uint32_t)(32 * c), v);
        tc::tmem_ld_32(up + lanes + (uint32_t)(32 * c), u);
        if (!p.tma || n % 8 != 0) {
            const int rows = min(32, e.M - row0);
            scale_and_bias_any<O>(v, sx, e.sg, e.bg, col, n, lane);
            scale_and_bias_any<O>(u, sx, e.su, e.bu, col, n, lane);
            if (e.Zg != nullptr)
                store_rows_any<O>(stage, lane, e.Zg, e.ldg, e.vec, row0, rows, col, n, v);
            if (e.Zu != nullptr)
                store_rows_any<O>(stage, lane, e.Zu, e.ldu, e.vec, row0, rows, col, n, u);
            gate_all<O>(v, u, e.act);
            store_rows_any<O>(stage, lane, e.H, e.ldh, e.vec, row0, rows, col, n, v);
            continue;
        }
        scale_and_bias32<O>(v, sx, e.sg, e.bg, col, n);
        scale_and_bias32<O>(u, sx, e.su, e.bu, col, n);
        if (keep && n == 32) {
            if (e.Zg != nullptr) stage_row<O>(stage, lane, v);
            if (e.Zu != nullptr) stage_row<O>(stage + 2048u, lane, u);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (e.Zg != nullptr) tma_store(map.Z, stage, col, row0);
                if (e.Zu != nullptr) tma_store(map.Z2, stage + 2048u, col, row0);
                tc::bulk_commit_group();
            }
        } else if (keep && in) {
            if (e.Zg != nullptr) store_row8s<O>(e.Zg, e.ldg, row, col, n, v);
            if (e.Zu != nullptr) store_row8s<O>(e.Zu, e.ldu, row, col, n, u);
        }
        gate_all<O>(v, u, e.act);
        if (n < 32) {
            if (in) store_row8s<O>(e.H, e.ldh, row, col, n, v);
            continue;
        }
        if (keep) {
            if (lane == 0) tc::bulk_wait_group_read<0>();
            __syncwarp();
        }
        stage_row<O>(stage, lane, v);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store(map.Y, stage, col, row0);
            tc::bulk_commit_group();
        }
    }
}

template <Form FORM, int CTAS, int BN, class O, bool SPLIT, class E>
__device__ __forceinline__ void linear_tc_body(const Maps &map, const Params<E> &p) {
    using S = Shape<CTAS, BN, SPLIT>;
    constexpr int STAGES = FORM == kGated ? kMostStages : S::STAGES, ACCS = S::ACCS;
    constexpr int BARS = 2 * STAGES + 2 * ACCS + 1;
    static_assert(BARS * 8 + 8 <= 256, "barrier area");
    constexpr bool CLUSTER = CTAS == 2 || SPLIT;
    // output columns of a tile; gated ones any multiple of 8 up to OUT (weights stored K x N:
    // OUT)
    constexpr int OUT = FORM == kGated ? BN / 2 : BN;
    constexpr bool ANY_OUT = FORM == kGated;
    const int out = ANY_OUT ? p.out : OUT;
    // Such a tile's stages are as large as its rows and outputs need, and as many as fit the
    // ring's place: 64 x 4096 x 4096 bf16 in tiles of 32 outputs was held by the 48 KB of
    // weights that whole tiles' stages had in flight (18.6 us, 16.4 so).
    constexpr int RING = S::STAGES * S::STAGE;
    const int a_tile = ANY_OUT ? p.a_tile : S::A_TILE, sub = ANY_OUT ? p.sub : S::SUB;
    const int stage_bytes = ANY_OUT ? S::KS * sub : S::STAGE;
    const int stages = ANY_OUT ? p.stages : S::STAGES;
    using Ring = typename std::conditional<ANY_OUT, tc::AnyRing, tc::Ring<S::STAGES>>::type;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = tc::smem_u32_generic(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw_addr & 1023)) & 1023);
    const uint32_t ring = tc::smem_u32_generic(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::STAGES * S::STAGE + S::STAGING);
    const uint32_t full0 = tc::smem_u32_generic(bars);
    const uint32_t empty0 = full0 + 8 * STAGES;
    const uint32_t accf0 = empty0 + 8 * STAGES;   // accumulator b holds a finished tile
    const uint32_t acce0 = accf0 + 8 * ACCS;      // accumulator b has been drained
    const uint32_t done_bar = acce0 + 8 * ACCS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + BARS);
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
        for (int s = 0; s < stages; ++s) {
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
        tc::tma_prefetch_desc(map.A);
        tc::tma_prefetch_desc(map.B);
        if constexpr (FORM == kSum) tc::tma_prefetch_desc(map.A2);
        if constexpr (FORM != kPlain) tc::tma_prefetch_desc(map.B2);
    }
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (CTAS == 2) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int bk = p.fp8 ? 128 : 64;
    // the boxes that bring B's rows of this CTA for columns tile tn and K block kb:
    // f(map, offset in the tile, coordinates)
    auto boxes_of_b = [&](int tn, int kb, auto f) {
        [[maybe_unused]] const CUtensorMap *b = map.B;
        if constexpr (FORM == kSum) {
            if (kb >= p.kblocks1) {
                b = map.B2;
                kb -= p.kblocks1;
            }
        }
        const int k0 = kb * bk;
        if constexpr (FORM == kGated) {
            // one matrix's rows in the even CTA, the other's in the odd one; both in
            // a CTA on its own
            const int n0 = tn * out;
#pragma unroll
            for (int h = 0; h < 3 - CTAS; ++h) {
                const CUtensorMap *w = (CTAS == 2 ? half : h) ? map.B2 : map.B;
                const int at = h * out * kRowBytes;
                if (p.b_kmajor) {
                    f(w, at, k0, n0);
                } else {
#pragma unroll
                    for (int c = 0; c < OUT / 64; ++c) f(w, at + c * kBox, n0 + 64 * c, k0);
                }
            }
        } else {
            const int n0 = tn * BN + half * S::BROWS;
            if (p.b_kmajor) {
                f(b, 0, k0, n0);
            } else {
#pragma unroll
                for (int c = 0; c < S::BROWS / 64; ++c) f(b, c * kBox, n0 + 64 * c, k0);
            }
        }
    };
    if (warp == 2 && ntiles > 0 && tc::elect_one()) {
        // the weights of the first stages into L2 while earlier work ends (L2 is where
        // that work's writes go, so nothing stale is read): a block of norm, 4096 ->
        // 8192 and back of 64 rows 39.2 -> 38.4 us in bf16, 28.8 -> 27.8 in 8 bits
        int tm, tn;
        raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first, tm, tn);
        for (int kb = kb0; kb < min(kb1, kb0 + S::KS * stages); ++kb)
            boxes_of_b(tn, kb, [&](const CUtensorMap *w, int, int c0, int c1) {
                tma_prefetch(w, c0, c1);
            });
    }
    __syncwarp();
    chain_begin(p.chain);   // nothing below reads or writes global memory before earlier work has finished

    if (warp == 0) {
        if (tc::elect_one()) {
            // ---------------- TMA producer: this CTA's rows of A and B
            const int b_bytes = ANY_OUT ? (3 - CTAS) * out * kRowBytes : S::B_TILE;
            const uint32_t tx = (uint32_t)(CTAS * (p.a_bytes + b_bytes));
            const uint32_t fulls = CTAS == 2 ? cluster_addr(full0, leader) : full0;
            Ring r(stages);
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                int tm, tn;
                raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first + i * stride, tm, tn);
                const int m0 = (tm * CTAS + half) * BM;
                for (int kb = kb0; kb < kb1; kb += S::KS) {
                    if (r.used == stages && !tc::wait(empty0 + 8 * r.s, r.parity ^ 1, abort_flag)) {
                        stop = true;
                        break;
                    }
                    const uint32_t fb = fulls + 8 * r.s;
                    const int subs = min(S::KS, kb1 - kb);
                    if (half == 0) tc::mbar_arrive_expect_tx(full0 + 8 * r.s, tx * subs);
#pragma unroll
                    for (int j = 0; j < S::KS; ++j) {
                        if (j >= subs) break;
                        const uint32_t st = ring + r.s * stage_bytes + j * sub;
                        const CUtensorMap *a = map.A;
                        int ka = kb + j;
                        if constexpr (FORM == kSum) {
                            if (ka >= p.kblocks1) {
                                a = map.A2;
                                ka -= p.kblocks1;
                            }
                        }
                        const int k0 = ka * bk;
                        if (p.a_kmajor) {
                            tma_load<CTAS>(st, a, fb, k0, m0);
                        } else {
#pragma unroll
                            for (int c = 0; c < BM / 64; ++c)
                                tma_load<CTAS>(st + c * kBox, a, fb, m0 + 64 * c, k0);
                        }
                        boxes_of_b(tn, kb + j, [&](const CUtensorMap *w, int at, int c0, int c1) {
                            tma_load<CTAS>(st + a_tile + at, w, fb, c0, c1);
                        });
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
            Ring r(stages);
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
                        const uint32_t st = ring + r.s * stage_bytes + j * sub;
                        const uint64_t ad = p.a_kmajor ? tc::kmajor_desc<128>(st) : mnmajor_desc(st);
                        const uint64_t bd = p.b_kmajor ? tc::kmajor_desc<128>(st + a_tile)
                                                       : mnmajor_desc(st + a_tile);
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
        if (reads_global(p.epi)) chain_fence(p.chain);   // through L1
        const int q = warp & 3, side = (warp - 2) >> 2;
        const uint32_t stage = ring + RING + (uint32_t)((warp - 2) * kStage);
        for (int i = 0; i < ntiles; ++i) {
            const int b = i % ACCS, u = i / ACCS;
            int tm, tn;
            raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first + i * stride, tm, tn);
            const int m0 = (tm * CTAS + half) * BM;
            // a side's columns: half of them, in blocks of 32 for gated tiles
            const int wide = ANY_OUT ? (out + 63) / 64 * 32 : OUT / 2;
            const int n0 = tn * out + side * wide, end = min(p.epi.N, tn * out + min(out, (side + 1) * wide));
            if constexpr (FORM == kGated)
                prefetch_terms<O>(p.epi, lane, n0, end);
            else
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
            } else if constexpr (FORM == kGated) {
                const uint32_t gate = tmem + (uint32_t)(b * BN + side * wide);
                finish_gated_rows<OUT / 64, O>(p, map, gate, gate + (uint32_t)out, q, lane, m0, n0,
                                               end, stage);
            } else {
                finish_rows<BN / 2, O, FORM == kSum>(p, map.Y, map.Z, acc, q, lane, m0, n0, stage);
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
        const int n0 = tn * out;
        if constexpr (FORM == kGated) {
            if (parts == 2) join_gated<2, CTAS, BN, O>(p.epi, ring, part, half, m0, n0, rows, out);
            if (parts == 4) join_gated<4, CTAS, BN, O>(p.epi, ring, part, half, m0, n0, rows, out);
            if (parts == 8) join_gated<8, CTAS, BN, O>(p.epi, ring, part, half, m0, n0, rows, out);
        } else {
            if (parts == 2) join_parts<2, CTAS, BN, O>(p.epi, ring, part, half, m0, n0, rows);
            if (parts == 4) join_parts<4, CTAS, BN, O>(p.epi, ring, part, half, m0, n0, rows);
            if (parts == 8) join_parts<8, CTAS, BN, O>(p.epi, ring, part, half, m0, n0, rows);
        }
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
inline bool operand_map(CUtensorMap *map, const TcOperand &o, int type, int rows, int K,
                        int box_rows) {
    return o.kmajor ? make_map(map, o.base, type, o.ld, K, rows, kRowBytes, box_rows,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B)
                    : make_map(map, o.base, type, o.ld, rows, K, kRowBytes, 64,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// A result that leaves in blocks of 32 columns by TMA store.
inline bool out_map(CUtensorMap *map, const void *base, int type, int64_t ld, int N, int M) {
    return make_map(map, base, type, ld, N, M, 64, 32, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// What the three forms' launches fill in alike: sizes, orientations, the piece.
// N: features of all matrices of a tile's columns (kGated: twice the outputs).
// Returns the rows of A's box.
template <int CTAS, int BN, class E>
int fill_params(Params<E> &p, int type, int M, int N, int K, bool a_kmajor, bool b_kmajor,
                const Piece &piece, int chain) {
    const int bk = kRowBytes / dtype_size(type);
    p.kblocks = p.kblocks1 = (K + bk - 1) / bk;
    p.tiles_m = (M + CTAS * BM - 1) / (CTAS * BM);
    p.tiles_n = (N + BN - 1) / BN;
    p.group_m = raster_group();
    p.a_kmajor = a_kmajor;
    p.b_kmajor = b_kmajor;
    // few rows: a box no higher than the rows (the tile's other rows are
    // whatever the stage held; they are computed and not stored)
    const int a_rows = M < BM ? (M + 7) / 8 * 8 : BM;
    p.a_bytes = a_kmajor ? a_rows * kRowBytes : BM * kRowBytes;
    p.idesc = instruction_desc(type, CTAS * BM, BN, a_kmajor, b_kmajor);
    p.fp8 = type == SGEMM_E4M3;
    p.error = device_error_word();
    p.chain = chain;
    p.tile0 = piece.tile0;
    p.tiles = piece.tiles;
    return a_rows;
}

template <class K>
cudaError_t configure(K kernel, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

}  // namespace ltc
}  // namespace sgemm
