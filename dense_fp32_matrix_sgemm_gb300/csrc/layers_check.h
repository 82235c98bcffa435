// What the layer operators' entry points share (layers_api.cu, block_api.cu): argument checks,
// the placing of operands that TMA cannot read, the epilogue of a plain product.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include <cuda_runtime.h>

#include "layers.h"

namespace sgemm {

int record_error(int code, const char *msg);   // api.cu
int require_device();

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxLd = (int64_t)1 << 37;   // byte strides stay below a tensor map's 2^40

inline int fail(int code, const char *fmt, ...) {
    char msg[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return record_error(code, msg);
}

inline bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline bool float_type(int t) { return t == SGEMM_F32 || t == SGEMM_BF16 || t == SGEMM_F16; }

inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }

inline int check_sizes(int64_t a, int64_t b, int64_t c, const char *names) {
    if (a < 0 || b < 0 || c < 0 || a > kMaxDim || b > kMaxDim || c > kMaxDim)
        return fail(SGEMM_EINVAL_DIM, "%s = %lld, %lld, %lld: each must be 0 .. 2^30", names,
                    (long long)a, (long long)b, (long long)c);
    return SGEMM_OK;
}

// A matrix argument: present where `need` says so, aligned to its elements,
// with a leading dimension of at least `cols`.
inline int check_matrix(const char *name, const void *p, int64_t ld, int64_t cols, int size, bool need) {
    const int64_t least = cols > 1 ? cols : 1;
    if (p == nullptr) {
        if (need) return fail(SGEMM_EINVAL_PTR, "%s is NULL", name);
        return SGEMM_OK;
    }
    if (ld < least || ld > kMaxLd)
        return fail(SGEMM_EINVAL_LD, "leading dimension of %s is %lld: must be %lld .. 2^37", name,
                    (long long)ld, (long long)least);
    if (!aligned(p, (uintptr_t)size))
        return fail(SGEMM_EINVAL_PTR, "%s is not %d-byte aligned", name, size);
    return SGEMM_OK;
}

#define CHECK(call)                  \
    do {                             \
        const int st_ = (call);      \
        if (st_ != SGEMM_OK) return st_; \
    } while (0)

inline int launched(cudaError_t e) {
    if (e != cudaSuccess)
        return fail(SGEMM_ELAUNCH, "kernel launch failed: %s", cudaGetErrorString(e));
    return SGEMM_OK;
}

inline int check_workspace(void *ws, uint64_t have, size_t need) {
    if (need > 0 && (ws == nullptr || !aligned(ws, 256) || have < need))
        return fail(SGEMM_EWORKSPACE, "workspace %p of %llu bytes: need %llu bytes, 256-byte aligned",
                    ws, (unsigned long long)have, (unsigned long long)need);
    return SGEMM_OK;
}

// A tensor-core operand of rows x cols as stored: whether TMA can read it
// where it lies, and the leading dimension (elements) and bytes of its copy
// with 128-byte rows where it cannot.
inline bool tma_ok(const void *p, int64_t ld, int size) { return aligned(p, 16) && ld * size % 16 == 0; }
inline int64_t padded_ld(int64_t cols, int size) { return (cols * size + 127) / 128 * 128 / size; }
inline size_t copy_bytes(const void *p, int64_t ld, int64_t rows, int64_t cols, int size) {
    return tma_ok(p, ld, size) ? 0 : round256((size_t)rows * padded_ld(cols, size) * size);
}

// The copy itself where one is needed, at *ws (advanced past it).
inline cudaError_t place(const void *&p, int64_t &ld, int64_t rows, int64_t cols, int size, char *&ws,
                  cudaStream_t s) {
    if (tma_ok(p, ld, size)) return cudaSuccess;
    const int64_t to = padded_ld(cols, size);
    const cudaError_t e = launch_repack(p, ld * size, rows, cols * size, size, ws, to * size, s);
    p = ws;
    ld = to;
    ws += round256((size_t)rows * to * size);
    return e;
}

inline int vector_width(int type, const LayerEpi &e) {
    const int size = dtype_size(type);
    auto all = [&](int n) {
        const uintptr_t bytes = (uintptr_t)(n * size);
        // bias and scales: 16-byte accesses at most
        const uintptr_t few = bytes < 16 ? bytes : 16;
        return aligned(e.Y, bytes) && e.ldy % n == 0 && aligned(e.bias, few) &&
               aligned(e.sw, n == 16 ? 16 : 4) &&
               (e.Z == nullptr || (aligned(e.Z, bytes) && e.ldz % n == 0)) &&
               (e.R == nullptr || (aligned(e.R, bytes) && e.ldr % n == 0));
    };
    return size == 2 && all(16) ? 16 : all(4) ? 4 : 1;
}

inline LayerEpi plain_epi(int type, void *Y, int64_t ldy, int64_t M, int64_t N) {
    LayerEpi e = {};
    e.Y = Y;
    e.ldy = ldy;
    e.M = (int)M;
    e.N = (int)N;
    e.act = SGEMM_ACT_NONE;
    e.type = type;
    e.vec = vector_width(type, e);
    return e;
}

}  // namespace sgemm
