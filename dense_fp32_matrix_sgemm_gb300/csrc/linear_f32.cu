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
//   linear_f32_kernel is linear_tc_kernel's pipeline on them: a stage holds 64
//     of K of the six tiles, and its 24 MMAs use each tile two or four times.
// The tensor cores add into their accumulator with a rounding towards zero, so
// a long sum there would collect errors of one sign.  Here an accumulator
// takes one stage: the five small terms first, while it is small, then a0 b0
// (four updates at full size), and the epilogue warps add it to running sums in
// registers with ordinary fp32 adds while the other accumulator fills.
// Measured against 64 bits: relative error @ERR@.
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
    static constexpr int STAGE = kPlanes * (A_TILE + B_TILE);
    static constexpr int STAGING = SPLIT ? 0 : kEpiWarps * kStage;
    static constexpr int STAGES = (kSmem - 1024 - 256 - STAGING) / STAGE;
    static constexpr int SLOTS = 2;   // accumulators, one stage's sum each
    static constexpr int TMEM_COLS = SLOTS * BN;
    static constexpr int BARS = 2 * STAGES + 2 * SLOTS + 1;
    static constexpr int SMEM = STAGES * STAGE + STAGING + 1024 + 256;
    static_assert(STAGES >= 2, "a stage loads while another is multiplied");
    static_assert(TMEM_COLS <= 512, "tensor memory");
    static_assert(BARS * 8 + 8 <= 256, "barrier area");
    static_assert(!SPLIT || BM * BN * 4 <= STAGES * STAGE, "a part of a tile fits the ring");
};

struct Params {
    LayerEpi epi;
    int kblocks;
    int tiles_m, tiles_n, group_m;
    int a_kmajor, b_kmajor;
    int a_bytes;        // bytes one plane of A brings to a CTA's stage
    uint32_t idesc;
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

// Roles, barriers and schedules as linear_tc_kernel; "accumulator full" and
// "empty" are per stage of K instead of per tile, counted across tiles.
template <int CTAS, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
linear_f32_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ Params p) {
    using S = Shape<CTAS, BN, SPLIT>;
    constexpr int STAGES = S::STAGES, SLOTS = S::SLOTS, COLS = BN / 2;
    constexpr bool CLUSTER = CTAS == 2 || SPLIT;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = tc::smem_u32_generic(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw_addr & 1023)) & 1023);
    const uint32_t ring = tc::smem_u32_generic(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * S::STAGE + S::STAGING);
    const uint32_t full0 = tc::smem_u32_generic(bars);
    const uint32_t empty0 = full0 + 8 * STAGES;
    const uint32_t accf0 = empty0 + 8 * STAGES;   // accumulator b holds a finished stage
    const uint32_t acce0 = accf0 + 8 * SLOTS;     // accumulator b has been drained
    const uint32_t done_bar = acce0 + 8 * SLOTS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + S::BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CLUSTER ? (int)cluster_rank() : 0;
    const int half = CTAS == 2 ? rank & 1 : 0;
    const int leader = CTAS == 2 ? rank & ~1 : rank;
    const uint16_t mask = (uint16_t)(3u << leader);
    const int total = p.tiles_m * p.tiles_n;
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
    pdl_trigger();
    pdl_wait();   // nothing below touches global memory before the planes are complete

    if (warp == 0) {
        if (tc::elect_one()) {
            // ---------------- TMA producer
            const uint32_t tx = (uint32_t)(CTAS * kPlanes * (p.a_bytes + S::B_TILE));
            const uint32_t fulls = CTAS == 2 ? cluster_addr(full0, leader) : full0;
            tc::Ring<STAGES> r;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                int tm, tn;
                raster(p.tiles_m, p.tiles_n, p.group_m, first + i * stride, tm, tn);
                const int m0 = (tm * CTAS + half) * BM, n0 = tn * BN + half * S::BROWS;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (r.used == STAGES &&
                        !tc::wait(empty0 + 8 * r.s, r.parity ^ 1, abort_flag)) {
                        stop = true;
                        break;
                    }
                    const uint32_t fb = fulls + 8 * r.s;
                    const int k0 = kb * kBk;
                    if (half == 0) tc::mbar_arrive_expect_tx(full0 + 8 * r.s, tx);
#pragma unroll
                    for (int pl = 0; pl < kPlanes; ++pl) {
                        const uint32_t a = ring + r.s * S::STAGE + pl * S::A_TILE;
                        const uint32_t b = ring + r.s * S::STAGE + kPlanes * S::A_TILE +
                                           pl * S::B_TILE;
                        if (p.a_kmajor) {
                            tma_load3<CTAS>(a, &tmA, fb, k0, m0, pl);
                        } else {
#pragma unroll
                            for (int c = 0; c < BM / 64; ++c)
                                tma_load3<CTAS>(a + c * kBox, &tmA, fb, m0 + 64 * c, k0, pl);
                        }
                        if (p.b_kmajor) {
                            tma_load3<CTAS>(b, &tmB, fb, k0, n0, pl);
                        } else {
#pragma unroll
                            for (int c = 0; c < S::BROWS / 64; ++c)
                                tma_load3<CTAS>(b + c * kBox, &tmB, fb, n0 + 64 * c, k0, pl);
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
            tc::Ring<SLOTS> q;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                for (int kb = 0; kb < nk; ++kb) {
                    if ((q.used == SLOTS &&
                         !tc::wait(acce0 + 8 * q.s, q.parity ^ 1, abort_flag)) ||
                        !tc::wait(full0 + 8 * r.s, r.parity, abort_flag)) {
                        stop = true;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t acc = tmem + (uint32_t)(q.s * BN);
                    const uint32_t st = ring + r.s * S::STAGE;
                    // the smallest terms first, a0 b0 last
                    constexpr int ta[6] = {2, 0, 1, 1, 0, 0}, tb[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
                    for (int t = 0; t < 6; ++t) {
                        const uint32_t a = st + ta[t] * S::A_TILE;
                        const uint32_t b = st + kPlanes * S::A_TILE + tb[t] * S::B_TILE;
                        const uint64_t ad = p.a_kmajor ? tc::kmajor_desc<128>(a) : mnmajor_desc(a);
                        const uint64_t bd = p.b_kmajor ? tc::kmajor_desc<128>(b) : mnmajor_desc(b);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma<CTAS, false>(acc, ad + kk * astep, bd + kk * bstep, p.idesc,
                                             (t | kk) ? 1u : 0u);
                    }
                    commit<CTAS>(empty0 + 8 * r.s, mask);
                    commit<CTAS>(accf0 + 8 * q.s, mask);
                    r.next();
                    q.next();
                }
            }
            commit<CTAS>(done_bar, mask);   // tracks every MMA issued above, also on abort
        }
    } else {
        // ---------------- epilogue: this CTA's rows, half of the columns a warp
        const int q = warp & 3, side = (warp - 2) >> 2;
        const uint32_t stage = ring + STAGES * S::STAGE + (uint32_t)((warp - 2) * kStage);
        tc::Ring<SLOTS> slot;
        bool stop = false;
        for (int i = 0; i < ntiles && !stop; ++i) {
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
            int tm, tn;
            raster(p.tiles_m, p.tiles_n, p.group_m, first + i * stride, tm, tn);
            const int row0 = (tm * CTAS + half) * BM + 32 * q, n0 = tn * BN + side * COLS;
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
                    __syncwarp();   // the previous block has been read
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        tc::st_shared_v4(stage + (uint32_t)lane * 128u +
                                             ((uint32_t)(j ^ (lane & 7)) << 4),
                                         run[32 * c + 4 * j], run[32 * c + 4 * j + 1],
                                         run[32 * c + 4 * j + 2], run[32 * c + 4 * j + 3]);
                    __syncwarp();
                    finish_staged<float>(p.epi, stage, lane, row0, rows, n0 + 32 * c + lane);
                }
            }
            __syncwarp();
        }
    }
    __syncwarp();

    tc::fence_before_sync();
    __syncthreads();
    if constexpr (SPLIT) {
        // every CTA of the cluster passes the barriers, an aborted one too
        cluster_sync();
        int tm, tn;
        raster(p.tiles_m, p.tiles_n, p.group_m, first, tm, tn);
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
};

// Two values as the three planes' pairs.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&w)[3]) {
    const float x0 = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
    const float y0 = __uint_as_float(__float_as_uint(y) & 0xffff0000u);
    const float rx = x - x0, ry = y - y0;   // exact
    w[0] = (__float_as_uint(x) >> 16) | (__float_as_uint(y) & 0xffff0000u);
    w[1] = pack2<__nv_bfloat16>(rx, ry);
    const float2 m = unpack2<__nv_bfloat16>(w[1]);
    w[2] = pack2<__nv_bfloat16>(rx - m.x, ry - m.y);
}

// CTAs [0, job[0].blocks) take the first operand, the rest the second; 8
// columns a thread with 16-byte accesses where the rows allow it, else 2.
__global__ void __launch_bounds__(256) split3_kernel(const SplitArgs a) {
    pdl_trigger();
    pdl_wait();
    const int which = (int)blockIdx.x < a.job[0].blocks ? 0 : 1;
    const SplitJob j = which ? a.job[1] : a.job[0];
    const int64_t block = (int64_t)blockIdx.x - (which ? a.job[0].blocks : 0);
    const int64_t plane = j.rows * j.ldp;
    const int w = j.vec ? 8 : 2;
    const int per_row = (j.cols + w - 1) / w;
    const int64_t total = j.rows * per_row;
    for (int64_t i = block * 256 + threadIdx.x; i < total; i += (int64_t)j.blocks * 256) {
        const int64_t r = i / per_row;
        const int c = (int)(i - r * per_row) * w;
        const float *x = j.X + r * j.ld + c;
        __nv_bfloat16 *out = j.out + r * j.ldp + c;
        if (j.vec) {   // cols is a multiple of 8
            const float4 u = __ldg(reinterpret_cast<const float4 *>(x));
            const float4 v = __ldg(reinterpret_cast<const float4 *>(x) + 1);
            uint32_t p[4][3];
            split_pair(u.x, u.y, p[0]);
            split_pair(u.z, u.w, p[1]);
            split_pair(v.x, v.y, p[2]);
            split_pair(v.z, v.w, p[3]);
#pragma unroll
            for (int pl = 0; pl < 3; ++pl)
                *reinterpret_cast<uint4 *>(out + pl * plane) =
                    make_uint4(p[0][pl], p[1][pl], p[2][pl], p[3][pl]);
        } else {
            uint32_t p[3];
            split_pair(__ldg(x), c + 1 < j.cols ? __ldg(x + 1) : 0.f, p);
#pragma unroll
            for (int pl = 0; pl < 3; ++pl)   // (the planes' rows are padded to 64)
                *reinterpret_cast<uint32_t *>(out + pl * plane) = p[pl];
        }
    }
}

// ------------------------------------------------------------------ host side

int64_t plane_ld(int64_t cols) { return (cols + 63) / 64 * 64; }

// Planes as [3][rows][cols], rows plane_ld(cols) apart: boxes as linear_tc's
// operands, one plane a load.  The maps end at the operand's own sizes, so the
// rows past K of an MN-major plane are zeros and not the next plane's.
bool plane_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const int64_t ld = plane_ld(cols);
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
cudaError_t launch(const F32Planes &A, const F32Planes &B, int K, const LayerEpi &epi, int parts,
                   int most, cudaStream_t s) {
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
    CUtensorMap tmA, tmB;
    if (!plane_map(&tmA, A.planes, A.rows, A.cols, A.kmajor ? a_rows : 64) ||
        !plane_map(&tmB, B.planes, B.rows, B.cols, B.kmajor ? S::BROWS : 64))
        return cudaErrorInvalidValue;
    const long long tiles = (long long)p.tiles_m * p.tiles_n;
    const long long ctas = SPLIT ? tiles * CTAS * parts : CTAS * (tiles < most ? tiles : most);
    Config c(ctas, S::SMEM, SPLIT ? CTAS * parts : CTAS, s);
    return cudaLaunchKernelEx(&c.cfg, linear_f32_kernel<CTAS, BN, SPLIT>, tmA, tmB, p);
}

}  // namespace f32
}  // namespace ltc

size_t f32_planes_bytes(int64_t rows, int64_t cols) {
    return ((size_t)ltc::f32::kPlanes * rows * ltc::f32::plane_ld(cols) * 2 + 255) / 256 * 256;
}

// Planes of one or two matrices, one launch; `out` at 256-byte boundaries.
cudaError_t launch_f32_split(const F32Operand *x, int count, cudaStream_t s) {
    using namespace ltc::f32;
    SplitArgs a = {};
    int blocks = 0;
    for (int i = 0; i < count; ++i) {
        SplitJob &j = a.job[i];
        j.X = x[i].X;
        j.out = static_cast<__nv_bfloat16 *>(x[i].planes);
        j.ld = x[i].ld;
        j.ldp = plane_ld(x[i].cols);
        j.rows = x[i].rows;
        j.cols = (int)x[i].cols;
        j.vec = x[i].cols % 8 == 0 && x[i].ld % 4 == 0 &&
                reinterpret_cast<uintptr_t>(x[i].X) % 16 == 0;
        const int w = j.vec ? 8 : 2;
        const int64_t need = (j.rows * ((j.cols + w - 1) / w) + 255) / 256;
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

// The tile and schedule by cost, as linear_tc's; a stage's 24 MMAs take
// @COST@.
cudaError_t launch_linear_f32(const F32Planes &A, const F32Planes &B, int K, const LayerEpi &epi,
                              cudaStream_t s) {
    using namespace ltc;
    Capacity cap;
    cudaError_t e = capacity(cap);
    if (e != cudaSuccess) return e;
    const int kblocks = (K + f32::kBk - 1) / f32::kBk;
    struct {
        int ctas, bn, parts;
        double us;
    } best = {0, 0, 0, 1e30};
    auto consider = [&](int ctas, int bn, int parts) {
        const long long tiles = (long long)((epi.M + ctas * BM - 1) / (ctas * BM)) *
                                ((epi.N + bn - 1) / bn);
        const int room = cap.of(ctas * parts);
        if (parts > 1 && (tiles > room || kblocks < 2 * parts)) return;
        const double stage = ctas == 2 ? 1.7 : bn == 128 ? 1.1 : 0.8;
        double us = (double)((tiles + room - 1) / room) * ((kblocks + parts - 1) / parts) * stage +
                    (ctas == 2 ? 7.5 : 6.0);
        if (parts > 1)
            us += 1.0 + (ctas == 2 ? 5.0 : 3.0 * bn / 128) * (epi.M < BM ? epi.M : BM) / BM;
        if (us < best.us) best = {ctas, bn, parts, us};
    };
    consider(2, 256, 1);
    consider(1, 64, 1);
    consider(1, 128, 1);
    for (int parts = 2; parts <= 8; parts *= 2) {
        if (parts <= 4) consider(2, 256, parts);
        consider(1, 128, parts);
        consider(1, 64, parts);
    }
    if (best.parts > 1) {
        if (best.ctas == 2) return f32::launch<2, 256, true>(A, B, K, epi, best.parts, 0, s);
        return best.bn == 128 ? f32::launch<1, 128, true>(A, B, K, epi, best.parts, 0, s)
                              : f32::launch<1, 64, true>(A, B, K, epi, best.parts, 0, s);
    }
    if (best.ctas == 2) return f32::launch<2, 256, false>(A, B, K, epi, 1, cap.of(2), s);
    return best.bn == 128 ? f32::launch<1, 128, false>(A, B, K, epi, 1, cap.sms, s)
                          : f32::launch<1, 64, false>(A, B, K, epi, 1, cap.sms, s);
}

}  // namespace sgemm
