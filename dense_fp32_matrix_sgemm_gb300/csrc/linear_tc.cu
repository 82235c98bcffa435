// The linear layer's product on the tensor cores: 16-bit or e4m3 operands,
// fp32 accumulation in tensor memory, the layer's epilogue on the way out.
//
//   D[row, col] = sum_k A(row, k) B(col, k)
//
// tcgen05.mma bounds it where all three sizes are large (2 M N K flops), HBM
// where one of them is small.  A CTA computes 128 x BN tiles with warps in
// three roles:
//   warp 0, lane 0: TMA producer: 128 bytes of K of A's and B's rows a stage,
//                   128-byte swizzle, a ring that runs on across tiles;
//   warp 1, lane 0: MMA issuer (M128 N=BN, 32 bytes of K an instruction);
//                   warp 1 owns tensor memory;
//   warps 2-5:      epilogue: TMEM lane quarter warp % 4, 64 columns at a time
//                   through the warp's own swizzled shared block, so global
//                   accesses are 16 bytes a lane and whole 128-byte row pieces.
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
constexpr int kThreads = 192;       // producer, MMA issuer, 4 epilogue warps
constexpr int kRowBytes = 128;      // of K in a stage
constexpr int kBox = 8192;          // MN-major box: 64 k x 128 bytes

template <int BN, bool SPLIT>
struct Shape {
    static constexpr int A_TILE = BM * kRowBytes;
    static constexpr int B_TILE = BN * kRowBytes;
    static constexpr int STAGE = A_TILE + B_TILE;
    static constexpr int STAGES = 192 * 1024 / STAGE;
    static constexpr int STAGING = 4 * 8192;   // an epilogue warp's 32 x 64 fp32 block
    static constexpr int ACCS = SPLIT ? 1 : 2;
    static constexpr int TMEM_COLS = ACCS * BN;
    static constexpr int BARS = 2 * STAGES + 2 * ACCS + 1;
    static constexpr int SMEM = STAGES * STAGE + STAGING + 1024 + 256;
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

__device__ __forceinline__ float4 ld_shared_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
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

// Finishes the 32 tile rows of TMEM lane quarter q, all columns.  Each 64
// columns pass through the warp's block at `stage` (256-byte rows; 16-byte
// chunk c of row r at c ^ (r & 7)): written a row a lane, read back as four
// rows an instruction, eight columns a lane.  The lane's two chunks are read
// in an order that keeps a quarter-warp on distinct banks.
template <int BN, class O>
__device__ __forceinline__ void finish_rows(const LayerEpi &e, uint32_t acc, int q, int lane,
                                            int m0, int n0, uint32_t stage) {
    const int row0 = m0 + 32 * q;
    if (row0 >= e.M) return;
    const uint32_t lane_base = acc + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
    for (int c = 0; c < BN / 64 && n0 + 64 * c < e.N; ++c) {
        __syncwarp();   // the previous block has been read
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[32];
            tc::tmem_ld_32(lane_base + (uint32_t)(64 * c + 32 * h), v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                tc::st_shared_v4(stage + (uint32_t)lane * 256u +
                                     ((uint32_t)((8 * h + j) ^ (lane & 7)) << 4),
                                 v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
        __syncwarp();
        const int l = lane & 7, odd = l >> 2;
        const int col = n0 + 64 * c + 8 * l;
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            const uint32_t base = stage + (uint32_t)r * 256u;
            const float4 a = ld_shared_v4(base + ((uint32_t)((2 * l + odd) ^ (r & 7)) << 4));
            const float4 b = ld_shared_v4(base + ((uint32_t)((2 * l + 1 - odd) ^ (r & 7)) << 4));
            const float4 lo = odd ? b : a, hi = odd ? a : b;
            const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            if (row0 + r < e.M && col < e.N) finish<O, 8>(e, row0 + r, col, v);
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
    const uint32_t staging = ring + STAGES * S::STAGE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * S::STAGE + S::STAGING);
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
            tc::mbar_init(acce0 + 8 * b, 4);   // one arrival an epilogue warp
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
        if (lane == 0) {
            // ---------------- TMA producer
            const int bk = p.fp8 ? 128 : 64;
            const uint32_t tx = (uint32_t)(p.a_bytes + S::B_TILE);
            long long g = 0;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                int tm, tn;
                raster(p, first + i * stride, tm, tn);
                const int m0 = tm * BM, n0 = tn * BN;
                for (int kb = kb0; kb < kb1; ++kb, ++g) {
                    const int s = (int)(g % STAGES);
                    if (g >= STAGES &&
                        !tc::mbar_wait(empty0 + 8 * s, (int)((g / STAGES) & 1) ^ 1, abort_flag)) {
                        stop = true;
                        break;
                    }
                    if (*abort_flag) {
                        stop = true;
                        break;
                    }
                    const uint32_t st = ring + s * S::STAGE, fb = full0 + 8 * s;
                    tc::mbar_arrive_expect_tx(fb, tx);
                    const int k0 = kb * bk;
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
                }
            }
            if (*abort_flag) {
                // the latest fill of every stage lands before the CTA exits
                for (long long f = (g > STAGES ? g - STAGES : 0); f < g; ++f) {
                    const int s = (int)(f % STAGES);
                    const long long t0 = clock64();
                    while (!tc::mbar_try_wait(full0 + 8 * s, (int)((f / STAGES) & 1)) &&
                           clock64() - t0 < tc::kWaitLimitCycles) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer
            const uint64_t astep = p.a_kmajor ? 2 : 128, bstep = p.b_kmajor ? 2 : 128;
            long long g = 0;
            bool stop = false;
            for (int i = 0; i < ntiles && !stop; ++i) {
                const int b = i % ACCS, u = i / ACCS;
                if (i >= ACCS && !tc::mbar_wait(acce0 + 8 * b, (u - 1) & 1, abort_flag)) break;
                tc::fence_after_sync();
                const uint32_t acc = tmem + (uint32_t)(b * BN);
                for (int kb = 0; kb < nk; ++kb, ++g) {
                    const int s = (int)(g % STAGES);
                    if (!tc::mbar_wait(full0 + 8 * s, (int)((g / STAGES) & 1), abort_flag)) {
                        stop = true;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t st = ring + s * S::STAGE;
                    const uint64_t ad = p.a_kmajor ? tc::kmajor_desc<128>(st) : mnmajor_desc(st);
                    const uint64_t bd = p.b_kmajor ? tc::kmajor_desc<128>(st + S::A_TILE)
                                                   : mnmajor_desc(st + S::A_TILE);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t more = (kb | kk) ? 1u : 0u;
                        if (p.fp8)
                            mma_f8(acc, ad + kk * astep, bd + kk * bstep, p.idesc, more);
                        else
                            mma_f16(acc, ad + kk * astep, bd + kk * bstep, p.idesc, more);
                    }
                    tc::mma_commit(empty0 + 8 * s);
                }
                if (!stop) tc::mma_commit(accf0 + 8 * b);
            }
            tc::mma_commit(done_bar);   // tracks every MMA issued above, also on abort
        }
    } else {
        // ---------------- epilogue
        const int q = warp & 3;
        for (int i = 0; i < ntiles; ++i) {
            const int b = i % ACCS, u = i / ACCS;
            const bool ok = tc::mbar_wait(accf0 + 8 * b, u & 1, abort_flag);
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
                    for (int c = 0; c < BN / 32; ++c) {
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
                finish_rows<BN, O>(p.epi, acc, q, lane, tm * BM, tn * BN,
                                   staging + (uint32_t)(warp - 2) * 8192u);
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

uint32_t instruction_desc(int type, int bn, bool a_kmajor, bool b_kmajor) {
    const uint32_t fmt = type == SGEMM_BF16 ? 1u : 0u;   // f16 and e4m3: 0
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_kmajor ? 0u : 1u) << 15) |
           ((b_kmajor ? 0u : 1u) << 16) | ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
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
    p.idesc = instruction_desc(type, BN, A.kmajor, B.kmajor);
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
    // waves of one tile an SM; a 256-wide tile costs about 1.7 128-wide ones
    const double wide = 1.7 * (double)((tiles(256) + sms - 1) / sms);
    const double narrow = (double)((tiles(128) + sms - 1) / sms);
    return wide <= narrow ? launch<256, O, false>(type, A, B, K, epi, 1, sms, s)
                          : launch<128, O, false>(type, A, B, K, epi, 1, sms, s);
}

}  // namespace ltc

cudaError_t launch_linear_tc(int in_type, const TcOperand &A, const TcOperand &B, int K,
                             const LayerEpi &epi, cudaStream_t s) {
    return epi.type == SGEMM_BF16 ? ltc::dispatch<__nv_bfloat16>(in_type, A, B, K, epi, s)
                                  : ltc::dispatch<__half>(in_type, A, B, K, epi, s);
}

}  // namespace sgemm
