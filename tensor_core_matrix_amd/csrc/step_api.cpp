// C ABI of the operators of a step that drafts (pages and slots, residual norm, 4-bit weights,
// attention of drafted tokens): argument validation and dispatch, in the order of layer_api.cpp.
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include <hip/hip_runtime.h>

#include "../../include/tcm.h"
#include "layer_checks.h"
#include "step_internal.h"
#include "tcm_host.h"

namespace {

using namespace tcm;

// ---- residual norm --------------------------------------------------------------

// T rows of D elements, ld apart; es bytes an element.
tcm_status check_rows(const void* p, int64_t ld, int64_t T, int64_t D, int64_t es) {
    if (!p) return TCM_ERR_NULL_POINTER;
    if (T > 1 && (ld < D || !stride_ok(T, ld))) return TCM_ERR_INVALID_SHAPE;
    if (!aligned16(p) || (T > 1 && ld * es % 16 != 0)) return TCM_ERR_MISALIGNED;
    return TCM_OK;
}

int64_t step(int64_t T, int64_t ld) { return T > 1 ? ld : 0; }

tcm_status check_norm(int64_t T, int64_t D, const void* weight, tcm_dtype weight_dtype, tcm_dtype dtype) {
    if (!half_type(dtype) || (weight && weight_dtype != TCM_F32 && weight_dtype != dtype))
        return TCM_ERR_UNSUPPORTED_DTYPE;
    if (T < 0 || D < 1) return TCM_ERR_INVALID_SHAPE;
    if (T > kMaxRows || D > kMaxNormDim) return TCM_ERR_UNSUPPORTED_SHAPE;
    return TCM_OK;
}

tcm_status add_rms_norm(const void* X, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                        tcm_dtype weight_dtype, float eps, void* sum, int64_t lds, void* Out,
                        int64_t ldo, uint8_t* scale, int64_t T, int64_t D, tcm_dtype dtype, NormOut out, void* stream) {
    tcm_status s = check_norm(T, D, weight, weight_dtype, dtype);
    if (s != TCM_OK || T == 0) return s;
    const int64_t oes = out == kNormF32 ? 4 : out == kNormMx ? 1 : 2;
    if ((s = check_rows(X, ldx, T, D, 2)) != TCM_OK) return s;
    if (residual && (s = check_rows(residual, ldr, T, D, 2)) != TCM_OK) return s;
    if (sum && (s = check_rows(sum, lds, T, D, 2)) != TCM_OK) return s;
    if ((s = check_rows(Out, ldo, T, D, oes)) != TCM_OK) return s;
    if (out == kNormMx && !scale) return TCM_ERR_NULL_POINTER;
    if (D % (out == kNormMx ? 32 : 8) != 0 || !aligned16(weight)) return TCM_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.x = X;
    a.r = residual;
    a.w = weight;
    a.sum = sum;
    a.out = Out;
    a.scale = scale;
    a.ldx = step(T, ldx);
    a.ldr = step(T, ldr);
    a.lds = step(T, lds);
    a.ldo = step(T, ldo);
    a.eps = eps;
    a.inv_d = 1.0f / (float)D;
    a.T = (int32_t)T;
    a.D = (int32_t)D;
    a.w_f32 = weight_dtype == TCM_F32;
    return launched(launch_add_rms_norm(a, (int32_t)dtype, out, (hipStream_t)stream));
}

// ---- attention of drafted tokens ----------------------------------------------------

// Rows of a workgroup (tree_attn.h): the tokens of one sequence times the query heads of a key-value head
int64_t tree_rows(int64_t G, int64_t D, int64_t max_nodes) {
    const int64_t n = max_nodes * G;
    return n <= 16 ? 16 : n <= 64 || D > 128 ? 64 : 128;
}
int64_t tree_blocks(int64_t G, int64_t D, int64_t max_nodes) {
    const int64_t n = cdiv(max_nodes * G, tree_rows(G, D, max_nodes));
    return n > 0 ? n : 1;
}
// Workgroups of a call whose blocks of rows number at most `units`, of at most `span` keys each: one a tile of
// the largest size, up to kTreeGroups.  A block of one tile is not split.
int64_t tree_groups(int64_t units, int64_t span, int64_t round) {
    const int64_t tiles = cdiv(span, round) > 0 ? cdiv(span, round) : 1;
    return units > kTreeGroups / tiles ? kTreeGroups : units * tiles;
}
int64_t tree_workspace(int64_t groups, int64_t rows, int64_t D, int64_t span, int64_t round) {
    return span > round ? groups * (2 * rows * (D + 2) * 4 + (int64_t)sizeof(TreeSplit)) : 0;
}

tcm_status check_tree_sizes(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_nodes, int64_t max_len) {
    if (B < 0 || Hq < 0 || Hk < 0 || D < 1 || max_nodes < 0 || max_len < 0) return TCM_ERR_INVALID_SHAPE;
    if ((Hq > 0 && Hk == 0) || (Hk > 0 && Hq % Hk != 0)) return TCM_ERR_INVALID_SHAPE;
    if (B > kMaxHeads || Hq > kMaxHeads || D > kMaxHeadDim || D % 8 != 0 || max_len > kMaxRows || max_nodes > kMaxRows ||
        (Hk > 0 && max_nodes * (Hq / Hk) > kMaxRows))
        return TCM_ERR_UNSUPPORTED_SHAPE;
    return TCM_OK;
}

int64_t norm_groups(int64_t T) { return T < kNormBwdGroups ? T : kNormBwdGroups; }

}  // namespace

extern "C" {

tcm_status tcm_cache_plan(int32_t* lengths, const int32_t* change, int32_t* block_table,
                          int64_t table_stride, int64_t table_width, int64_t B, int64_t pages,
                          int64_t page_size, int32_t* free_pages, int64_t capacity,
                          int32_t* free_count, int32_t* starts, int32_t* slots, int32_t* positions,
                          int64_t T, int32_t* missing, void* stream) {
    if (B < 0 || table_width < 0 || pages < 0 || page_size < 1 || capacity < 0 || T < 0 ||
        (B > 1 && table_stride < table_width))
        return TCM_ERR_INVALID_SHAPE;
    if (B > kMaxHeads || page_size > (int64_t(1) << 20) || pages > INT32_MAX / page_size ||
        table_width > kMaxRows / page_size || T > kMaxRows || capacity > INT32_MAX || (B > 1 && table_stride > INT32_MAX))
        return TCM_ERR_UNSUPPORTED_SHAPE;
    if (!starts || !free_count || (B > 0 && (!lengths || !change)) || (B > 0 && table_width > 0 && !block_table) ||
        (capacity > 0 && !free_pages))
        return TCM_ERR_NULL_POINTER;
    DeviceInfo dev;
    tcm_status s;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    PlanArgs a;
    memset(&a, 0, sizeof(a));
    a.lengths = lengths;
    a.change = change;
    a.table = block_table;
    a.table_stride = B > 1 ? table_stride : 0;
    a.stack = free_pages;
    a.count = free_count;
    a.starts = starts;
    a.slots = slots;
    a.positions = positions;
    a.missing = missing;
    a.B = (int32_t)B;
    a.width = (int32_t)table_width;
    a.pages = (int32_t)pages;
    a.page_size = (int32_t)page_size;
    a.capacity = (int32_t)capacity;
    a.T = (int32_t)T;
    a.page_shift = shift_of(page_size);
    return launched(launch_cache_plan(a, (hipStream_t)stream));
}

tcm_status tcm_add_rms_norm(const void* X, int64_t ldx, const void* residual, int64_t ldr,
                            const void* weight, tcm_dtype weight_dtype, float eps, void* sum,
                            int64_t lds, void* Out, int64_t ldo, int64_t T, int64_t D,
                            tcm_dtype dtype, tcm_dtype out_dtype, void* stream) {
    if (out_dtype != dtype && out_dtype != TCM_F32) return TCM_ERR_UNSUPPORTED_DTYPE;
    return add_rms_norm(X, ldx, residual, ldr, weight, weight_dtype, eps, sum, lds, Out, ldo, nullptr, T, D, dtype,
                        out_dtype == dtype ? kNormHalf : kNormF32, stream);
}

tcm_status tcm_add_rms_norm_mx_fp8(const void* X, int64_t ldx, const void* residual, int64_t ldr,
                                   const void* weight, tcm_dtype weight_dtype, float eps,
                                   void* sum, int64_t lds, void* Out, void* scale, int64_t T,
                                   int64_t D, tcm_dtype dtype, void* stream) {
    return add_rms_norm(X, ldx, residual, ldr, weight, weight_dtype, eps, sum, lds, Out, cdiv(D, 16) * 16,
                        (uint8_t*)scale, T, D, dtype, kNormMx, stream);
}

tcm_status tcm_add_rms_norm_bwd_workspace(int64_t T, int64_t D, int64_t* bytes) {
    if (!bytes) return TCM_ERR_NULL_POINTER;
    if (T < 0 || D < 1) return TCM_ERR_INVALID_SHAPE;
    if (T > kMaxRows || D > kMaxNormDim) return TCM_ERR_UNSUPPORTED_SHAPE;
    *bytes = norm_groups(T) * D * 4;
    return TCM_OK;
}

tcm_status tcm_add_rms_norm_bwd(const void* dOut, int64_t lddo, const void* dsum, int64_t ldds,
                                const void* S, int64_t lds, const void* weight,
                                tcm_dtype weight_dtype, float eps, void* dX, int64_t lddx,
                                float* dweight, int64_t T, int64_t D, tcm_dtype dtype,
                                void* workspace, int64_t workspace_bytes, void* stream) {
    tcm_status s = check_norm(T, D, weight, weight_dtype, dtype);
    if (s != TCM_OK || (T == 0 && !dweight)) return s;
    if (T > 0) {
        if ((s = check_rows(dOut, lddo, T, D, 2)) != TCM_OK || (s = check_rows(S, lds, T, D, 2)) != TCM_OK ||
            (s = check_rows(dX, lddx, T, D, 2)) != TCM_OK)
            return s;
        if (dsum && (s = check_rows(dsum, ldds, T, D, 2)) != TCM_OK) return s;
    }
    if (D % 8 != 0 || !aligned16(weight)) return TCM_ERR_MISALIGNED;
    if (dweight && T > 0) {
        if (!workspace) return TCM_ERR_NULL_POINTER;
        if (!aligned16(workspace)) return TCM_ERR_MISALIGNED;
        if (workspace_bytes < norm_groups(T) * D * 4) return TCM_ERR_WORKSPACE;
    }
    DeviceInfo dev;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.x = S;
    a.r = dsum;
    a.dy = dOut;
    a.w = weight;
    a.out = dX;
    a.ldx = step(T, lds);
    a.ldr = step(T, ldds);
    a.lddy = step(T, lddo);
    a.ldo = step(T, lddx);
    a.eps = eps;
    a.inv_d = 1.0f / (float)D;
    a.T = (int32_t)T;
    a.D = (int32_t)D;
    a.w_f32 = weight_dtype == TCM_F32;
    a.partial = (float*)workspace;
    a.dw = dweight;
    a.groups = (int32_t)norm_groups(T);
    return launched(launch_add_rms_norm_bwd(a, (int32_t)dtype, (hipStream_t)stream));
}

tcm_status tcm_gemm_w4(const void* X, int64_t ldx, const void* W, const void* scales,
                       const void* zeros, void* Out, int64_t ldo, int64_t M, int64_t N, int64_t K,
                       int64_t group, tcm_dtype elem, tcm_dtype dtype, tcm_dtype out_dtype,
                       void* stream) {
    if (!half_type(dtype) || !(out_dtype == dtype || out_dtype == TCM_F32) || (elem != TCM_U4 && elem != TCM_E2M1))
        return TCM_ERR_UNSUPPORTED_DTYPE;
    const bool e2m1 = elem == TCM_E2M1;
    if (M < 0 || N < 0 || K < 0 || group < 1 || (M > 1 && (ldx < K || ldo < N))) return TCM_ERR_INVALID_SHAPE;
    if (M > kMaxRows || N > kMaxRows || K > kMaxK || K % 32 != 0 || group % 32 != 0 || K % group != 0 ||
        (e2m1 && group != 32) || (M > 1 && (ldx > kMaxLd || ldo > INT32_MAX)))
        return TCM_ERR_UNSUPPORTED_SHAPE;
    // a launch's workgroups in the one and the other direction, and its threads
    if (cdiv(M, 64) > 65535 || cdiv(M, 64) * cdiv(N, 16) > UINT32_MAX / 512) return TCM_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return TCM_OK;
    if (!Out || (K > 0 && (!X || !W || !scales))) return TCM_ERR_NULL_POINTER;
    if (e2m1 && zeros) return TCM_ERR_INVALID_ARGUMENT;
    const auto off = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (!aligned16(X) || !aligned16(W) || (M > 1 && ldx % 8 != 0) || (!e2m1 && off(scales, 2)) ||
        off(Out, out_dtype == TCM_F32 ? 4 : 2))
        return TCM_ERR_MISALIGNED;
    DeviceInfo dev;
    tcm_status s;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    W4Args a;
    memset(&a, 0, sizeof(a));
    a.x = X;
    a.w = (const uint8_t*)W;
    a.scales = scales;
    a.zeros = (const uint8_t*)zeros;
    a.out = Out;
    a.ldo = step(M, ldo);
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.ldx = (int32_t)step(M, ldx);
    a.gchunks = (int32_t)(group / 32);
    a.gshift = shift_of(a.gchunks);
    a.groups = (int32_t)(K / group);
    return launched(launch_gemm_w4(a, (int32_t)dtype, e2m1, out_dtype == TCM_F32, dev.cus, (hipStream_t)stream));
}

tcm_status tcm_paged_tree_attention_workspace(int64_t B, int64_t Hq, int64_t Hk, int64_t D,
                                              int64_t max_nodes, int64_t max_len, int64_t* bytes) {
    if (!bytes) return TCM_ERR_NULL_POINTER;
    tcm_status s = check_tree_sizes(B, Hq, Hk, D, max_nodes, max_len);
    if (s != TCM_OK) return s;
    *bytes = 0;
    if (B == 0 || Hq == 0 || max_nodes == 0) return TCM_OK;
    // (tiles of E4M3 keys are at least as long; a window's first tile begins up to 31 keys early)
    const int64_t G = Hq / Hk, rows = tree_rows(G, D, max_nodes), round = tree_round(rows, D, 2);
    *bytes = tree_workspace(tree_groups(B * Hk * tree_blocks(G, D, max_nodes), max_len, round), rows, D, max_len, round);
    return TCM_OK;
}

tcm_status tcm_paged_tree_attention(const tcm_heads* q, const tcm_cache* cache,
                                    const int32_t* block_table, int64_t table_stride,
                                    const int32_t* lengths, int64_t max_len,
                                    const int32_t* starts, int64_t max_nodes, const uint64_t* tree,
                                    int64_t tree_words, const tcm_heads* out, float* lse, int64_t T,
                                    int64_t B, int64_t Hq, int64_t Hk, int64_t D, float scale,
                                    int64_t window, tcm_dtype dtype, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
    if (!half_type(dtype)) return TCM_ERR_UNSUPPORTED_DTYPE;
    tcm_status s = check_tree_sizes(B, Hq, Hk, D, max_nodes, max_len);
    if (s != TCM_OK) return s;
    if (T < 0 || window < 0 || table_stride < 0 || tree_words < 0 || (tree && tree_words < cdiv(max_nodes, 64)))
        return TCM_ERR_INVALID_SHAPE;
    if (T > kMaxRows || table_stride > INT32_MAX || (tree && tree_words > kMaxRows / 2)) return TCM_ERR_UNSUPPORTED_SHAPE;
    if ((s = check_cache(cache, dtype, Hk, D, false)) != TCM_OK) return s;
    if (cache->dtype == TCM_E4M3 && D % 16 != 0) return TCM_ERR_MISALIGNED;
    if (T == 0 || B == 0 || Hq == 0 || max_nodes == 0) return TCM_OK;
    if (!lengths || !starts || (table_stride > 0 && !block_table)) return TCM_ERR_NULL_POINTER;
    if ((s = check_heads(q, T, Hq)) != TCM_OK || (s = check_written(out, T, Hq, D)) != TCM_OK) return s;
    if (reinterpret_cast<uintptr_t>(tree) % 8 != 0) return TCM_ERR_MISALIGNED;
    // no page, no key
    if (cache->pages == 0) max_len = 0;
    const int64_t G = Hq / Hk, rows = tree_rows(G, D, max_nodes), blocks = tree_blocks(G, D, max_nodes);
    if (B * Hk > kMaxRows / blocks) return TCM_ERR_UNSUPPORTED_SHAPE;
    const bool e4m3 = cache->dtype == TCM_E4M3;
    const int64_t round = tree_round(rows, D, e4m3 ? 1 : 2), groups = tree_groups(B * Hk * blocks, max_len, round);
    const int64_t need = tree_workspace(groups, rows, D, max_len, round);
    if (need > 0) {
        if (!workspace) return TCM_ERR_NULL_POINTER;
        if (!aligned16(workspace)) return TCM_ERR_MISALIGNED;
        if (workspace_bytes < need) return TCM_ERR_WORKSPACE;
    }
    DeviceInfo dev;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    TreeArgs a;
    memset(&a, 0, sizeof(a));
    const int64_t es = e4m3 ? 1 : 2;
    a.q = view(q, T, Hq);
    a.out = view(out, T, Hq);
    a.kc = (const char*)cache->k;
    a.vc = (const char*)cache->v;
    a.k_page = step_bytes(cache->pages, cache->k_page_stride, es);
    a.k_tok = step_bytes(cache->page_size, cache->k_token_stride, es);
    a.k_head = step_bytes(Hk, cache->k_head_stride, es);
    a.v_page = step_bytes(cache->pages, cache->v_page_stride, es);
    a.v_tok = step_bytes(cache->page_size, cache->v_token_stride, es);
    a.v_head = step_bytes(Hk, cache->v_head_stride, es);
    a.table = block_table;
    a.table_stride = table_stride;
    a.lengths = lengths;
    a.starts = starts;
    a.tree = (const uint32_t*)tree;
    a.tree_words = tree ? (int32_t)(2 * tree_words) : 0;
    a.lse = lse;
    if (need > 0) {
        a.po = (float*)workspace;
        a.pml = a.po + groups * 2 * rows * D;
        a.split = (TreeSplit*)(a.pml + groups * 2 * rows * 2);
    }
    a.T = (int32_t)T;
    a.B = (int32_t)B;
    a.Hq = (int32_t)Hq;
    a.Hk = (int32_t)Hk;
    a.G = (int32_t)G;
    a.D = (int32_t)D;
    a.pages = (int32_t)cache->pages;
    a.page_size = (int32_t)cache->page_size;
    // With 2^s >= page_size the first power of two, m = floor(2^(31 + s) / page_size) + 1 is at most 2^(31 + s) /
    // page_size + 1, so n m is past n 2^(31 + s) / page_size by at most n < 2^31 <= 2^(31 + s) / page_size (and m <
    // 2^32): the quotient's whole part is right.
    int s2 = 0;
    while ((int64_t(1) << s2) < cache->page_size) ++s2;
    a.page_magic = (uint32_t)((uint64_t(1) << (31 + s2)) / (uint64_t)cache->page_size + 1);
    a.page_shift = 31 + s2;
    a.max_len = (int32_t)max_len;
    a.max_nodes = (int32_t)max_nodes;
    // A window that keeps no row from any key is none.  (A sequence may have more tokens than keys, so a chain's last
    // ones may be max_len + max_nodes places, at most 2^31, behind a key.)
    a.window = window >= max_len + max_nodes ? 0 : (int32_t)window;
    a.groups = (int32_t)groups;
    a.rows = (int32_t)rows;
    a.scale_log2 = scale * (e4m3 ? cache->k_scale : 1.0f) * 1.4426950408889634f;
    a.v_scale = e4m3 ? cache->v_scale : 1.0f;
    hipStream_t st = (hipStream_t)stream;
    return launched(dtype == TCM_BF16 ? launch_tree_attention_bf16(a, e4m3, st) : launch_tree_attention_f16(a, e4m3, st));
}

}  // extern "C"
