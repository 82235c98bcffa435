// Shared by the linear layer's tensor-core kernels (linear_tc.cu, linear_f32.cu):
// tile constants, PTX wrappers for one CTA and for pairs, the tile order, the
// joining of split tiles, tensor maps and launch attributes.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "device_utils.cuh"
#include "gemm_args.h"
#include "layer_math.cuh"
#include "layers.h"
#include "tc_issue.cuh"
#include "tc_utils.cuh"
#include "tma_encode.h"

namespace sgemm {
namespace ltc {

constexpr int BM = 128;             // rows of a CTA's tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kRowBytes = 128;      // of K in a stage
constexpr int kBox = 8192;          // MN-major box: 64 k x 128 bytes
constexpr int kSmem = 227 * 1024;
constexpr int kStage = 4096;        // an epilogue warp's staging block

// ------------------------------------------------------------------ PTX

// 2-D tiled load of the box at (c0, c1) into this CTA's shared memory,
// completing on `bar`: a barrier of this CTA, or (CTAS = 2, a shared::cluster
// address) of the pair's even CTA.  c0 (innermost) is a multiple of 16 bytes.
template <int CTAS>
__device__ __forceinline__ void tma_load(uint32_t dst, const void *tmap, uint32_t bar, int c0,
                                         int c1) {
    if constexpr (CTAS == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];"
            :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
            :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
}

// Asks for the box at (c0, c1) in L2.
__device__ __forceinline__ void tma_prefetch(const void *tmap, int c0, int c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];"
                 :: "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1) : "memory");
}

__device__ __forceinline__ void tma_store(const void *tmap, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                 :: "l"(reinterpret_cast<uint64_t>(tmap)), "r"(src), "r"(c0), "r"(c1)
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

template <int CTAS, bool FP8>
__device__ __forceinline__ void mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                    uint32_t idesc, uint32_t accumulate) {
#define SGEMM_MMA(group, kind)                                                                  \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                              \
                 "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}"    \
                 :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)            \
                 : "memory")
    if constexpr (CTAS == 1 && FP8) SGEMM_MMA("1", "f8f6f4");
    if constexpr (CTAS == 1 && !FP8) SGEMM_MMA("1", "f16");
    if constexpr (CTAS == 2 && FP8) SGEMM_MMA("2", "f8f6f4");
    if constexpr (CTAS == 2 && !FP8) SGEMM_MMA("2", "f16");
#undef SGEMM_MMA
}

// Arrive on `bar` (CTAS = 2: in both CTAs of the pair, `mask`) once every MMA
// issued so far by this thread has completed.
template <int CTAS>
__device__ __forceinline__ void commit(uint32_t bar, uint16_t mask) {
    if constexpr (CTAS == 1)
        tc::mma_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                     ".multicast::cluster.b64 [%0], %1;" :: "r"(bar), "h"(mask) : "memory");
}

template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t slot_smem, uint32_t ncols) {
    if constexpr (CTAS == 1) {
        tc::tmem_alloc(slot_smem, ncols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(slot_smem), "r"(ncols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CTAS>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    if constexpr (CTAS == 1)
        tc::tmem_dealloc(taddr, ncols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                     :: "r"(taddr), "r"(ncols) : "memory");
}

// The shared::cluster address of `addr` (shared::cta) in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Arrival on another CTA's barrier that publishes no memory: it says that this
// warp's loads from tensor memory have completed (each waits for its data).  With
// .release the warp first waits for all it has written and read, about 1700 clocks.
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];"
                 :: "r"(cluster_bar) : "memory");
}

// ------------------------------------------------------------------ tiles

// Tile t of a tiles_m x tiles_n grid, walked in groups of group_m tile rows
// (tiles that run together share operand panels in L2).
__device__ __forceinline__ void raster(int tiles_m, int tiles_n, int group_m, int t, int &tm,
                                       int &tn) {
    const int group = group_m * tiles_n;
    const int g = t / group;
    const int first = g * group_m;
    const int rows = min(tiles_m - first, group_m);
    const int r = t - g * group;
    tm = first + r % rows;
    tn = r / rows;
}

// Brings a row's piece of the residual into L2 while the tile's product runs: the
// epilogue waits for HBM otherwise, block after block (2049 x 3071 x 1537 f32 with
// a residual: 115.7 us, 113.7 so; 8192^3 e4m3 312, 301).
template <class O>
__device__ __forceinline__ void prefetch_residual(const LayerEpi &e, int row, int col, int cols) {
    if (e.R == nullptr || row >= e.M) return;
    const O *r = static_cast<const O *>(e.R) + row * e.ldr;
    for (int c = col; c < min(col + cols, e.N); c += 128 / (int)sizeof(O))
        prefetch_l2(r + c);
}

// The epilogue on the first `rows` rows (from row0 on) of a 32 x 32 fp32 block
// that the warp has staged at `stage` (16-byte chunk j of row r at chunk
// j ^ (r & 7) of its 128 bytes): a column a lane, U rows (8, 16) at a time, so
// each access is a whole row segment and U residual loads are in flight (one row
// at a time, an f32 layer of 2049 x 3071 outputs with a residual took 100 us
// more than without; with eight in flight 114, with sixteen 106).
template <class O, int U>
__device__ __forceinline__ void finish_staged(const LayerEpi &e, uint32_t stage, int lane, int row0,
                                              int rows, int col) {
    if (col >= e.N) return;
    ColumnTerms<O, 1> t;
    t.load(e, col);
#pragma unroll 1
    for (int r = 0; r < rows; r += U) {
        float x[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[i])
                         : "r"(stage + (uint32_t)(r + i) * 128u +
                               ((uint32_t)((lane >> 2) ^ (i & 7)) << 4) + (uint32_t)((lane & 3) * 4))
                         : "memory");
        finish_column<O, U>(e, t, row0 + r, rows - r, col, x);
    }
}

// This CTA's share of the rows of the tile that PARTS CTAs hold parts of, in
// their shared memory at `ring` (row r, 16-byte chunk c at c ^ (r & 7) of its
// BN * 4 bytes).  A lane keeps four columns of each half of the tile and walks
// rows, so the columns' terms are loaded once and what is left per row is
// 2 PARTS loads, the sums in K order and two 8-byte stores; the lanes of a load
// read consecutive chunks (half as many packets between SMs as with eight
// consecutive columns a lane).  U rows are in flight.  (Four columns a thread
// at a time, each with its own row and column arithmetic, took 9 us of a
// 256 x 256 tile where this takes 3.)
template <int PARTS, int CTAS, int BN, class O>
__device__ __forceinline__ void join_parts(const LayerEpi &e, uint32_t ring, int part, int half,
                                           int m0, int n0, int rows) {
    constexpr int LPR = BN / 8, RPW = 32 / LPR;   // lanes a row, rows a warp
    constexpr int STEP = kThreads / 32 * RPW * PARTS;
    constexpr int U = PARTS == 2 ? 4 : PARTS == 8 ? 1 : 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = lane % LPR;
    const int col[2] = {n0 + 4 * c, n0 + 4 * (c + LPR)};
    if (col[0] >= e.N) return;
    ColumnTerms<O, 4> t[2];
    t[0].load(e, col[0]);
    t[1].load(e, col[1]);
    uint32_t base[PARTS];
#pragma unroll
    for (int j = 0; j < PARTS; ++j) base[j] = cluster_addr(ring, CTAS * j + half);
    for (int r0 = (warp * PARTS + part) * RPW + lane / LPR; r0 < rows; r0 += U * STEP) {
        float4 x[U][2][PARTS];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * STEP;
            if (r >= rows) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = (uint32_t)(r * BN * 4) +
                                    ((uint32_t)((c + h * LPR) ^ (r & 7)) << 4);
#pragma unroll
                for (int j = 0; j < PARTS; ++j) x[u][h][j] = ld_cluster_v4(base[j] + at);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * STEP;
            if (r >= rows) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 s = x[u][h][0];
#pragma unroll
                for (int j = 1; j < PARTS; ++j) {
                    s.x += x[u][h][j].x;
                    s.y += x[u][h][j].y;
                    s.z += x[u][h][j].z;
                    s.w += x[u][h][j].w;
                }
                float v[4] = {s.x, s.y, s.z, s.w};
                if (col[h] < e.N) finish_group<O, 4>(e, t[h], m0 + r, col[h], v);
            }
        }
    }
}

// ------------------------------------------------------------------ host side

inline CUtensorMapDataType map_type(int type) {
    return type == SGEMM_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
           : type == SGEMM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
           : type == SGEMM_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                               : CU_TENSOR_MAP_DATA_TYPE_UINT8;
}

// A rows x cols row-major matrix read or written in boxes of box_bytes (128 or
// 64, with the swizzle of that span) x box_rows.
inline bool make_map(CUtensorMap *map, const void *base, int type, int64_t ld, int cols, int rows,
              int box_bytes, int box_rows, CUtensorMapL2promotion promote) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const int size = dtype_size(type);
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * size};
    const cuuint32_t box[2] = {(cuuint32_t)(box_bytes / size), (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, map_type(type), 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, promote,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline uint32_t instruction_desc(int type, int bm, int bn, bool a_kmajor, bool b_kmajor) {
    const uint32_t fmt = type == SGEMM_BF16 ? 1u : 0u;   // f16 and e4m3: 0
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_kmajor ? 0u : 1u) << 15) |
           ((b_kmajor ? 0u : 1u) << 16) | ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(bm >> 4) << 24);
}

// Launch attributes: programmatic dependent launch and, above 1, a cluster.
struct Config {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Config(long long ctas, int smem, int cluster, cudaStream_t s) {
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = cluster > 1 ? 2 : 1;
    }
};

// Clusters of 2, 4 and 8 CTAs of these kernels that the device holds at once
// (on GB300 76, 36 and 15: SMs come in groups that whole clusters do not fill).
struct Capacity {
    int sms, clusters[3];
    int of(int size) const { return size == 1 ? sms : clusters[size == 2 ? 0 : size == 4 ? 1 : 2]; }
    Capacity half() const { return {sms / 2, {clusters[0] / 2, clusters[1] / 2, clusters[2] / 2}}; }
};
cudaError_t capacity(Capacity &cap);   // linear_tc.cu

// Consecutive tiles in one launch: `parts` K parts each (1: whole tiles,
// walked by at most `room` CTAs or pairs).
struct Piece {
    int tile0, tiles, parts, room;
};

// Tiles of ctas * 128 x bn; a kernel is built for a few shapes.
struct TileShape {
    int ctas, bn;
};

// How a product is computed: tiles of one shape, in one launch, or (pairs) whole
// waves of tiles in one and the rest split in K in a second.
struct Plan {
    int shape = 0;
    int pieces = 0;
    Piece piece[2];
    double us = 1e30;
};

// The shapes and, in microseconds, what 128 bytes (f32: 64) of K of a tile take,
// what a launch takes besides, and the joining of the parts of a split tile of 128
// rows (next to 1 us a split launch).
template <int SHAPES>
struct Costs {
    TileShape shape[SHAPES];
    double stage[SHAPES], fixed[SHAPES], join[SHAPES];
};

template <int SHAPES>
Plan plan_tiles(int M, int N, int kblocks, const Capacity &cap, const Costs<SHAPES> &cost) {
    Plan best;
    const double rows = (M < BM ? M : BM) / (double)BM;
    // one split launch of `tiles` tiles; negative where it cannot run at once
    auto split = [&](int w, long long tiles, int parts) {
        const int ctas = cost.shape[w].ctas;
        if (tiles > cap.of(ctas * parts) || kblocks < 2 * parts) return -1.0;
        return ((kblocks + parts - 1) / parts) * cost.stage[w] + cost.fixed[w] + 1.0 +
               cost.join[w] * rows;
    };
    auto take = [&](double us, int w, Piece a, Piece b, int pieces) {
        if (us >= best.us) return;
        best.us = us;
        best.shape = w;
        best.piece[0] = a;
        best.piece[1] = b;
        best.pieces = pieces;
    };
    for (int w = 0; w < SHAPES; ++w) {
        const int ctas = cost.shape[w].ctas, bn = cost.shape[w].bn;
        const long long all = (long long)((M + ctas * BM - 1) / (ctas * BM)) * ((N + bn - 1) / bn);
        if (all > 0x7fffffff) continue;
        const int tiles = (int)all, room = cap.of(ctas);
        const long long waves = tiles / room;
        const int tail = (int)(tiles - waves * room);
        take((double)(waves + (tail > 0)) * kblocks * cost.stage[w] + cost.fixed[w], w,
             {0, tiles, 1, room}, {}, 1);
        for (int parts = 2; parts <= (ctas == 2 ? 4 : 8); parts *= 2) {
            const double whole = split(w, tiles, parts);
            if (whole > 0) take(whole, w, {0, tiles, parts, 0}, {}, 1);
            const double rest = ctas == 2 && waves > 0 && tail > 0 ? split(w, tail, parts) : -1;
            if (rest > 0)
                take((double)waves * kblocks * cost.stage[w] + cost.fixed[w] + rest, w,
                     {0, tiles - tail, 1, room}, {tiles - tail, tail, parts, 0}, 2);
        }
    }
    return best;
}

// Two products that each leave SMs idle take the time of the longer one when
// each is planned for half of the SMs; in turn, the second one's start is hidden
// by the first (about 4 us).  (Gradients of 500 x 777 x 1001 f32: 31.5 us in turn, 27.2 so; 1024 x 2048 x 2048
// bf16 27.9 and 23.7.)
template <int SHAPES>
bool side_by_side(const ProductSize &a, const ProductSize &b, int k_stage, const Capacity &cap,
                  const Costs<SHAPES> &cost) {
    auto us = [&](const ProductSize &p, const Capacity &c) {
        return plan_tiles(p.M, p.N, (p.K + k_stage - 1) / k_stage, c, cost).us;
    };
    const Capacity half = cap.half();
    if (half.clusters[0] < 1) return false;
    const double ha = us(a, half), hb = us(b, half);
    return (ha > hb ? ha : hb) < us(a, cap) + us(b, cap) - 4.0;
}

// f(w as a constant).
template <int W, int SHAPES, class F>
cudaError_t with_shape(int w, F &&f) {
    if constexpr (W < SHAPES)
        return w == W ? f(std::integral_constant<int, W>()) : with_shape<W + 1, SHAPES>(w, f);
    else
        return cudaErrorInvalidValue;
}

// launch(shape's index and split as constants, the piece, its place in the chain)
// for every piece of the plan.
template <int SHAPES, class F>
cudaError_t run_plan(const Costs<SHAPES> &, const Plan &plan, int chain, F &&launch) {
    if (plan.pieces == 0) return cudaErrorInvalidConfiguration;   // more than 2^31 tiles
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < plan.pieces && e == cudaSuccess; ++i) {
        const Piece &p = plan.piece[i];
        const int at = (i > 0 ? kChainPrev : chain & kChainPrev) |
                       (i + 1 < plan.pieces ? kChainNext : chain & kChainNext);
        e = with_shape<0, SHAPES>(plan.shape, [&](auto w) {
            return p.parts > 1 ? launch(w, std::true_type(), p, at)
                               : launch(w, std::false_type(), p, at);
        });
    }
    return e;
}

}  // namespace ltc
}  // namespace sgemm
