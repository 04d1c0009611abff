// Argument checks shared by the C ABI's translation units of the layer operators (host only).
#pragma once

#include <limits.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/tcm.h"
#include "layer_internal.h"

namespace tcm {

namespace {

constexpr int64_t kMaxK = int64_t(1) << 20;
constexpr int64_t kMaxLd = int64_t(1) << 21;   // 256 rows of it stay within 32 bits
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxHeads = 65535;
// elements; no device memory holds a larger step
constexpr int64_t kMaxStride = int64_t(1) << 40;

// 16 tokens of a page stay within 32 bits of bytes
constexpr int64_t kMaxTokenStride = int64_t(1) << 25;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool half_type(tcm_dtype d) { return d == TCM_F16 || d == TCM_BF16; }

inline tcm_status launched(hipError_t e) { return e == hipSuccess ? TCM_OK : TCM_ERR_HIP; }

// ---- views ----------------------------------------------------------------------

// A stride is not negative, and n steps of it (n >= 0) stay far within 64 bits of bytes.
// Where n <= 1 no step is taken, and any stride will do.
inline bool stride_ok(int64_t n, int64_t stride) {
    int64_t t;
    if (n <= 1) return true;
    return stride >= 0 && stride <= kMaxStride && !__builtin_mul_overflow(n, stride, &t) &&
           t < (int64_t(1) << 60);
}

inline tcm_status check_heads(const tcm_heads* v, int64_t T, int64_t H) {
    if (!v || !v->ptr) return TCM_ERR_NULL_POINTER;
    if (!stride_ok(T, v->token_stride) || !stride_ok(H, v->head_stride)) return TCM_ERR_INVALID_SHAPE;
    if (!aligned16(v->ptr) || (T > 1 && v->token_stride % 8 != 0) || (H > 1 && v->head_stride % 8 != 0))
        return TCM_ERR_MISALIGNED;
    return TCM_OK;
}

// A view that is written: its tokens and heads lie apart.
inline tcm_status check_written(const tcm_heads* v, int64_t T, int64_t H, int64_t D) {
    tcm_status s = check_heads(v, T, H);
    if (s != TCM_OK) return s;
    const int64_t ts = v->token_stride, hs = v->head_stride;
    if (T > 1 && H > 1) {
        // one of the two is the outer one and steps over the whole of the other
        const bool tokens_outer = hs >= D && ts >= (H - 1) * hs + D;
        const bool heads_outer = ts >= D && hs >= (T - 1) * ts + D;
        if (!tokens_outer && !heads_outer) return TCM_ERR_INVALID_SHAPE;
    } else if ((T > 1 && ts < D) || (H > 1 && hs < D)) {
        return TCM_ERR_INVALID_SHAPE;
    }
    return TCM_OK;
}

inline HeadView view(const tcm_heads* v, int64_t T, int64_t H) {
    return {v->ptr, T > 1 ? v->token_stride : 0, H > 1 ? v->head_stride : 0};
}

inline tcm_status check_cache(const tcm_cache* c, tcm_dtype dtype, int64_t Hk, int64_t D, bool written) {
    if (!c) return TCM_ERR_NULL_POINTER;
    if (c->dtype != dtype && c->dtype != TCM_E4M3) return TCM_ERR_UNSUPPORTED_DTYPE;
    if (c->pages < 0 || c->page_size < 1) return TCM_ERR_INVALID_SHAPE;
    const int64_t st[6] = {c->k_page_stride, c->k_token_stride, c->k_head_stride,
                           c->v_page_stride, c->v_token_stride, c->v_head_stride};
    const int64_t count[3] = {c->pages, c->page_size, Hk};
    for (int i = 0; i < 6; ++i)
        if (!stride_ok(count[i % 3], st[i])) return TCM_ERR_INVALID_SHAPE;
    if (written) {
        // every (page, place, head) its own D elements at least
        for (int i = 0; i < 6; i += 3) {
            if ((c->pages > 1 && st[i] < D) || (c->page_size > 1 && st[i + 1] < D) ||
                (Hk > 1 && st[i + 2] < D))
                return TCM_ERR_INVALID_SHAPE;
        }
    }
    if (c->pages > 0 && (!c->k || !c->v)) return TCM_ERR_NULL_POINTER;
    if (c->pages > INT32_MAX || c->page_size > (int64_t(1) << 20) ||
        (c->page_size > 1 && (c->k_token_stride > kMaxTokenStride || c->v_token_stride > kMaxTokenStride)))
        return TCM_ERR_UNSUPPORTED_SHAPE;
    const int64_t piece = c->dtype == TCM_E4M3 ? 16 : 8;
    for (int i = 0; i < 6; ++i)
        if (count[i % 3] > 1 && st[i] % piece != 0) return TCM_ERR_MISALIGNED;
    if (!aligned16(c->k) || !aligned16(c->v)) return TCM_ERR_MISALIGNED;
    return TCM_OK;
}

// A stride in bytes; none where there is no step of it.
inline int64_t step_bytes(int64_t n, int64_t stride, int64_t es) { return n > 1 ? stride * es : 0; }

// log2 of a power of two, -1 of any other page size
inline int32_t shift_of(int64_t page_size) {
    for (int32_t i = 0; i <= 20; ++i)
        if (page_size == int64_t(1) << i) return i;
    return -1;
}

}  // namespace

}  // namespace tcm
