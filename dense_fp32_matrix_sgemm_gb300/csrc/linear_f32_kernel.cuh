// The f32 product's kernel (described in linear_f32.cu) in its three forms:
// linear_f32.cu launches the plain one, gated_f32.cu the two others.
#pragma once

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

template <class E>
struct Params {
    E epi;
    int kblocks;
    int kblocks1;       // kSum: of the first product's K, where the second begins
    int out;            // kGated, pairs: outputs of a tile
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
template <Form FORM, int CTAS, int BN, bool SPLIT, class E>
__device__ __forceinline__ void linear_f32_body(const Maps &map, const Params<E> &p) {
    using S = Shape<CTAS, BN, SPLIT>;
    constexpr int RING = S::RING, SLOTS = S::SLOTS, COLS = BN / 2;
    // output columns of a tile; of pairs' gated ones any multiple of 8 up to OUT (weights stored
    // K x N: OUT)
    constexpr int OUT = FORM == kGated ? BN / 2 : BN;
    constexpr bool ANY_OUT = FORM == kGated && CTAS == 2;
    const int out = ANY_OUT ? p.out : OUT;
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
    chain_begin(p.chain);   // nothing below touches global memory before the planes are complete

    if (warp == 0) {
        if (tc::elect_one()) {
            // ---------------- TMA producer: a stage's planes in the issuer's order
            const uint32_t tx =
                (uint32_t)(CTAS * (p.a_bytes + (ANY_OUT ? out * kRowBytes : S::B_TILE)));
            const uint32_t fulls = CTAS == 2 ? cluster_addr(full0, leader) : full0;
            tc::Ring<RING> r;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                int tm, tn;
                raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first + i * stride, tm, tn);
                const int m0 = (tm * CTAS + half) * BM;
                for (int kb = kb0; kb < kb1 && !stop; ++kb) {
                    const CUtensorMap *ma = map.A, *mb = map.B;
                    int k0 = kb * kBk;
                    if constexpr (FORM == kSum) {
                        if (kb >= p.kblocks1) {
                            ma = map.A2;
                            mb = map.B2;
                            k0 -= p.kblocks1 * kBk;
                        }
                    }
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
                            tma_load3<CTAS>(a, ma, fb, k0, m0, order[j]);
                        } else {
#pragma unroll
                            for (int c = 0; c < BM / 64; ++c)
                                tma_load3<CTAS>(a + c * kBox, ma, fb, m0 + 64 * c, k0, order[j]);
                        }
                        if constexpr (FORM == kGated) {
                            // (the weights' places as in linear_tc_body)
                            const int n0 = tn * out;
#pragma unroll
                            for (int h = 0; h < 3 - CTAS; ++h) {
                                const CUtensorMap *w = (CTAS == 2 ? half : h) ? map.B2 : mb;
                                const uint32_t to = b + h * OUT * kRowBytes;
                                if (OUT < 64 || p.b_kmajor) {
                                    tma_load3<CTAS>(to, w, fb, k0, n0, order[j]);
                                } else {
#pragma unroll
                                    for (int c = 0; c < OUT / 64; ++c)
                                        tma_load3<CTAS>(to + c * kBox, w, fb, n0 + 64 * c, k0,
                                                        order[j]);
                                }
                            }
                        } else {
                            const int n0 = tn * BN + half * S::BROWS;
                            if (p.b_kmajor) {
                                tma_load3<CTAS>(b, mb, fb, k0, n0, order[j]);
                            } else {
#pragma unroll
                                for (int c = 0; c < S::BROWS / 64; ++c)
                                    tma_load3<CTAS>(b + c * kBox, mb, fb, n0 + 64 * c, k0,
                                                    order[j]);
                            }
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
        if (reads_global(p.epi)) chain_fence(p.chain);
        const int q = warp & 3, side = (warp - 2) >> 2;
        const uint32_t stage = ring + RING * S::PLANE + (uint32_t)((warp - 2) * kStage);
        tc::Ring<SLOTS> slot;
        bool stop = false;
        for (int i = 0; i < ntiles && !stop; ++i) {
            int tm, tn;
            raster(p.tiles_m, p.tiles_n, p.group_m, p.tile0 + first + i * stride, tm, tn);
            // a side's columns: half of them, in blocks of 16 for gated tiles
            const int wide = ANY_OUT ? (out + 31) / 32 * 16 : OUT / 2;
            const int row0 = (tm * CTAS + half) * BM + 32 * q, n0 = tn * out + side * wide;
            const int end = min(p.epi.N, tn * out + min(out, (side + 1) * wide));
            if constexpr (FORM != kGated) prefetch_residual<float>(p.epi, row0 + lane, n0, COLS);
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
                // (kGated: half of the side's columns are gates, half their factors)
                const uint32_t base = tmem + (uint32_t)(slot.s * BN + side * wide) +
                                      ((uint32_t)(32 * q) << 16);
#pragma unroll
                for (int b = 0; b < COLS / 16; ++b) {
                    float v[16];
                    const int at = FORM == kGated && b >= OUT / 32 ? out + 16 * b - OUT / 2 : 16 * b;
                    tc::tmem_ld_16(base + at, v);
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
                for (int j = 0; j < COLS / 4; ++j) {
                    const bool up = FORM == kGated && j >= OUT / 8;
                    const int at = side * (wide / 4) + (up ? j - OUT / 8 : j);
                    // (past a side's columns are the other one's, or none)
                    if (ANY_OUT && 4 * (up ? j - OUT / 8 : j) >= min(wide, out - side * wide)) continue;
                    tc::st_shared_v4(ring + (uint32_t)(r * BN * 4) +
                                         ((uint32_t)((at + (up ? out / 4 : 0)) ^ (r & 7)) << 4),
                                     run[4 * j], run[4 * j + 1], run[4 * j + 2], run[4 * j + 3]);
                }
            } else if constexpr (FORM == kGated) {
                // 16 outputs at a time, in a rolled loop (its code is fetched once): the first 16
                // gates and factors leave, the others move down
                const int rows = min(32, p.epi.M - row0);
#pragma unroll 1
                for (int c = 0; c < OUT / 32 && n0 + 16 * c < end; ++c) {
                    __syncwarp();   // the previous block has been read
                    stage_pair16(stage, lane, run, run + OUT / 2);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j + 16 < OUT / 2; ++j) {
                        run[j] = run[j + 16];
                        run[OUT / 2 + j] = run[OUT / 2 + j + 16];
                    }
                    finish_gated_staged<float, 8>(p.epi, stage, lane, row0, rows, n0 + 16 * c, end);
                }
            } else {
                const int rows = min(32, p.epi.M - row0);
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) {
                    if (n0 + 32 * c >= p.epi.N) break;
                    if (p.tma && n0 + 32 * c + 32 <= p.epi.N) {
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = run[32 * c + j];
                        store_row32(p.epi, map.Y, stage, lane, row0, n0 + 32 * c, v);
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
        const int n0 = tn * out;
        if constexpr (FORM == kGated) {
            if (parts == 2)
                join_gated<2, CTAS, BN, float>(p.epi, ring, part, half, m0, n0, rows, out);
            if (parts == 4)
                join_gated<4, CTAS, BN, float>(p.epi, ring, part, half, m0, n0, rows, out);
            if (parts == 8)
                join_gated<8, CTAS, BN, float>(p.epi, ring, part, half, m0, n0, rows, out);
        } else {
            if (parts == 2) join_parts<2, CTAS, BN, float>(p.epi, ring, part, half, m0, n0, rows);
            if (parts == 4) join_parts<4, CTAS, BN, float>(p.epi, ring, part, half, m0, n0, rows);
            if (parts == 8) join_parts<8, CTAS, BN, float>(p.epi, ring, part, half, m0, n0, rows);
        }
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

// ------------------------------------------------------------------ host side

// Planes as [3][rows][cols], rows f32_plane_ld(cols) apart: boxes as linear_tc's
// operands, one plane a load.  The maps end at the operand's own sizes, so the
// rows past K of an MN-major plane are zeros and not the next plane's.
inline bool plane_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int box_rows) {
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

// What the three forms' launches fill in alike (N: features of all matrices of a tile's
// columns).  Returns the rows of A's box.
template <int CTAS, int BN, class E>
int fill_params(Params<E> &p, int M, int N, int K, bool a_kmajor, bool b_kmajor, const Piece &piece,
                int chain) {
    p.kblocks = p.kblocks1 = (K + kBk - 1) / kBk;
    p.tiles_m = (M + CTAS * BM - 1) / (CTAS * BM);
    p.tiles_n = (N + BN - 1) / BN;
    p.group_m = raster_group();
    p.a_kmajor = a_kmajor;
    p.b_kmajor = b_kmajor;
    const int a_rows = M < BM ? (M + 7) / 8 * 8 : BM;
    p.a_bytes = a_kmajor ? a_rows * kRowBytes : BM * kRowBytes;
    p.idesc = instruction_desc(SGEMM_BF16, CTAS * BM, BN, a_kmajor, b_kmajor);
    p.tma = 0;
    p.error = device_error_word();
    p.chain = chain;
    p.tile0 = piece.tile0;
    p.tiles = piece.tiles;
    return a_rows;
}

// Whether a result leaves by TMA store; its map if so.
inline bool stores_by_tma(const LayerEpi &epi, CUtensorMap *tmY) {
    return epi.vec == 4 && epi.Z == nullptr &&
           (epi.act == SGEMM_ACT_NONE || epi.act == SGEMM_ACT_RELU) &&
           make_map(tmY, epi.Y, SGEMM_F32, epi.ldy, epi.N, epi.M, 128, 32,
                    CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// Costs of the shapes (see linear_f32.cu).
constexpr Costs<4> kCosts = {{{2, 256}, {2, 128}, {1, 64}, {1, 128}}, {1.66, 0.89, 0.78, 1.05},
                             {8.5, 8.0, 6.0, 6.0}, {5.0, 3.0, 1.5, 3.0}};

}  // namespace f32
}  // namespace ltc
}  // namespace sgemm
