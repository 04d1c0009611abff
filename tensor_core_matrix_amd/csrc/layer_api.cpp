// C ABI of the layer operators (adapters, norm and rotation of heads, paged
// attention): argument validation and dispatch, in the order of tcm_api.cpp:
// dtypes and enumerations, sizes, pointers, supported range, alignment, workspace.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <hip/hip_runtime.h>

#include "../../include/tcm.h"
#include "layer_checks.h"
#include "layer_internal.h"
#include "tcm_host.h"

namespace {

using namespace tcm;

// ---- norm and rotation -------------------------------------------------------------

tcm_status check_rope(const tcm_rope* r, tcm_dtype dtype, int64_t T, int64_t Hq, int64_t Hk) {
    if (!half_type(dtype)) return TCM_ERR_UNSUPPORTED_DTYPE;
    if (!r) return TCM_ERR_NULL_POINTER;
    if (r->layout != TCM_ROPE_HALF && r->layout != TCM_ROPE_INTERLEAVED) return TCM_ERR_INVALID_ARGUMENT;
    const bool weighted = r->norm && (r->q_weight || r->k_weight);
    if (weighted && r->weight_dtype != dtype && r->weight_dtype != TCM_F32) return TCM_ERR_UNSUPPORTED_DTYPE;
    if (T < 0 || Hq < 0 || Hk < 0 || r->head_dim < 1 || r->rot_dim < 0 || r->rot_dim > r->head_dim ||
        r->rot_dim % 2 != 0)
        return TCM_ERR_INVALID_SHAPE;
    if (T > kMaxRows || Hq > kMaxHeads || Hk > kMaxHeads || r->head_dim > kMaxHeadDim ||
        r->head_dim % 8 != 0)
        return TCM_ERR_UNSUPPORTED_SHAPE;
    if (T > 0 && Hq + Hk > 0 && r->rot_dim > 0 && (!r->positions || !r->inv_freq))
        return TCM_ERR_NULL_POINTER;
    if (weighted && (!aligned16(r->q_weight) || !aligned16(r->k_weight))) return TCM_ERR_MISALIGNED;
    return TCM_OK;
}

void fill_rope(RopeArgs* a, const tcm_rope* r, int64_t T, int64_t Hq, int64_t Hk) {
    memset(a, 0, sizeof(*a));
    a->pos = r->positions;
    a->inv_freq = r->inv_freq;
    a->wq = r->norm ? r->q_weight : nullptr;
    a->wk = r->norm ? r->k_weight : nullptr;
    a->eps = r->eps;
    a->factor = r->factor;
    a->T = (int32_t)T;
    a->Hq = (int32_t)Hq;
    a->Hk = (int32_t)Hk;
    a->D = (int32_t)r->head_dim;
    a->rot = (int32_t)r->rot_dim;
    a->norm = r->norm != 0;
    a->w_f32 = r->weight_dtype == TCM_F32;
    a->inv_d = 1.0f / (float)r->head_dim;
}

E4m3Scale scale_parts(float scale) {
    E4m3Scale s;
    int e = 0;
    s.m = frexpf(scale, &e);
    s.inv = 1.0f / s.m;
    s.top = 448.0f * fabsf(s.m);
    s.e = e;
    return s;
}

int64_t bwd_workspace(int64_t D) { return int64_t(kRopeBwdGrid) * 2 * D * 4; }

// ---- paged attention ----------------------------------------------------------------

// The split over the length.  Two ways to deal the work to workgroups of four waves:
//  * heads == 1: a chunk of one key-value head's keys, its tiles dealt to the
//    waves.  Chunks of 1024 keys, or fewer (256 at least) where that leaves fewer than
//    1024 workgroups: 64 sequences of up to 4096 keys took 100 us in chunks of 1024,
//    101 of 768 and 107 of 2048 (lengths differ: the last chunks idle the device);
//    32 of up to 8192 E4M3 keys 67, and 72 in chunks of 512 (each pays its first
//    reads' latency).
//  * heads == 4: the same chunk of four heads, one a wave, so that the
//    workgroup reads whole stretches of memory (a probe that only reads reaches
//    6.9 TB/s that way and 6.4 with a head a workgroup).  It is for few sequences with
//    work for every one of 256 compute units.  us this way and the other, 8 key-value
//    heads of 128: 1 sequence of 131072 keys (256 workgroups) 87 and 94, of 65536 (128)
//    62 and 52; 4 of 32768 (256) 87 and 93, of which three are shorter 64 and 64, of
//    16384 (128) 62 and 51; beyond four sequences both sides come near: 8 of 16384
//    (256) 87 and 93, 16 of up to 16384 (512) 118 and 109, 32 of up to 8192 123 and 118.
// A launch holds less than 2^32 threads, 256 a workgroup: where the chunks of very many
// sequences and heads would pass that, they are longer.
constexpr int64_t kMinChunk = 256, kChunk = 1024, kMostGroups = UINT32_MAX / 256;
struct Split {
    int64_t chunk, n, heads;
};
int64_t split_units(int64_t B, int64_t Hq, int64_t Hk) {
    const int64_t units = B * Hk * cdiv(Hq / Hk, 16);
    return units > 0 ? units : 1;
}
Split split_of(int64_t B, int64_t Hq, int64_t Hk, int64_t span) {
    Split s;
    s.heads = Hk % 4 == 0 && B <= 4 && B * (Hk / 4) * cdiv(span, kChunk) >= 256 ? 4 : 1;
    s.chunk = kChunk;
    if (s.heads == 1) {
        const int64_t c = cdiv(cdiv(span, cdiv(1024, split_units(B, Hq, Hk))), 128) * 128;
        s.chunk = c < kMinChunk ? kMinChunk : c < kChunk ? c : kChunk;
    }
    int64_t most = kMostGroups / split_units(B, Hq, Hk);
    if (most > kAttnMaxSplits) most = kAttnMaxSplits;
    if (most < 1) most = 1;
    if (cdiv(span, s.chunk) > most) s.chunk = cdiv(cdiv(span, most), 128) * 128;
    s.n = cdiv(span, s.chunk);
    if (s.n < 1) s.n = 1;
    return s;
}
// No split_of() of at most B sequences and this span has more chunks over all of them
// (0: none has more than one a sequence).  Either the chunks are the longest, or they
// are cut for 1024 workgroups over `units` a sequence: ceil(x / b) chunks of b
// sequences, x = ceil(1024 / units), are fewer than x + b, for b < x.
int64_t most_chunks(int64_t B, int64_t Hq, int64_t Hk, int64_t span) {
    const int64_t longest = cdiv(span, kChunk), shortest = cdiv(span, kMinChunk);
    const int64_t lo = longest < kAttnMaxSplits ? longest : kAttnMaxSplits;
    const int64_t hi = shortest < kAttnMaxSplits ? shortest : kAttnMaxSplits;
    const int64_t x = cdiv(1024, split_units(1, Hq, Hk));
    int64_t cut = x + (B < x ? B : x) - 1;
    if (cut > B * hi) cut = B * hi;
    if (hi <= 1) cut = 0;
    const int64_t whole = lo > 1 ? B * lo : 0;
    return cut > whole ? cut : whole;
}
// of so many chunks over all sequences
int64_t attn_workspace(int64_t chunks, int64_t Hq, int64_t D) { return chunks * Hq * (D + 2) * 4; }

tcm_status check_attn_sizes(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
    if (B < 0 || Hq < 0 || Hk < 0 || D < 1 || max_len < 0) return TCM_ERR_INVALID_SHAPE;
    if ((Hq > 0 && Hk == 0) || (Hk > 0 && Hq % Hk != 0)) return TCM_ERR_INVALID_SHAPE;
    if (B > kMaxHeads || Hq > kMaxHeads || D > kMaxHeadDim || D % 8 != 0 || max_len > kMaxRows)
        return TCM_ERR_UNSUPPORTED_SHAPE;
    return TCM_OK;
}

// ---- adapters ------------------------------------------------------------------------

// Parts of K in the adapters' first product, such that its workgroups -- one for
// each row with few rows, for each 16 rows with many -- are about 1024, four for every
// compute unit, whose reads' latency they hide from each other.  A part is at least
// 1024 values, a 128-deep piece for each of a workgroup's eight waves, and there are
// at most four (eight below 16 rows), the reads of t that the second product has
// under way at once.
int64_t lora_parts(int64_t M, int64_t K, int64_t* kpart) {
    const int64_t groups = M <= 256 ? M : cdiv(M, 16);
    int64_t n = groups > 0 ? 1024 / groups : 1;
    const int64_t most = M < 16 ? 8 : 4;
    if (n > most) n = most;
    if (n > K / 1024) n = K / 1024;
    if (n < 1) n = 1;
    *kpart = cdiv(cdiv(K, n), 1024) * 1024;
    if (*kpart < 1024) *kpart = 1024;
    n = cdiv(K, *kpart);
    return n > 0 ? n : 1;
}

// No lora_parts() of at most M rows and K values times its rows is more.  The parts that
// rows and K allow fall with the rows, in steps whose last rows are the most of each (15
// rows of up to eight parts, then 16 for every sixteenth of 1024 / n), and grow with K.
int64_t lora_most_rows(int64_t M, int64_t K) {
    auto rows = [&](int64_t last, int64_t n) {
        const int64_t fit = K / 1024 > 1 ? K / 1024 : 1;
        return (M < last ? M : last) * (n < fit ? n : fit);
    };
    int64_t most = rows(15, 8);
    for (int64_t n = 1; n <= 4; ++n) {
        const int64_t r = n > 1 ? rows(16 * (1024 / n), n) : M;
        if (r > most) most = r;
    }
    return most;
}

tcm_status check_lora_sizes(int64_t M, int64_t K, int64_t R) {
    if (M < 0 || K < 0 || R < 0) return TCM_ERR_INVALID_SHAPE;
    if (M > kMaxRows || K > kMaxK || R > kLoraMaxRank) return TCM_ERR_UNSUPPORTED_SHAPE;
    return TCM_OK;
}

}  // namespace

extern "C" {

tcm_status tcm_lora_workspace(int64_t M, int64_t K, int64_t R, int64_t* bytes) {
    if (!bytes) return TCM_ERR_NULL_POINTER;
    tcm_status s = check_lora_sizes(M, K, R);
    if (s != TCM_OK) return s;
    *bytes = lora_most_rows(M, K) * R * 4;
    return TCM_OK;
}

tcm_status tcm_lora_gemm_tn(const void* X, int64_t ldx, const void* W, const void* A,
                            const void* B, const int32_t* row_adapter, const int32_t* ranks,
                            const float* scales, void* Out, int64_t ldo, int64_t M, int64_t N,
                            int64_t K, int64_t L, int64_t R, tcm_dtype dtype, tcm_dtype out_dtype,
                            void* workspace, int64_t workspace_bytes, void* stream) {
    if (!half_type(dtype) || !(out_dtype == dtype || out_dtype == TCM_F32))
        return TCM_ERR_UNSUPPORTED_DTYPE;
    if (N < 0 || L < 0 || (M != 1 && (ldx < (K > 1 ? K : 1) || ldo < (N > 1 ? N : 1)))) return TCM_ERR_INVALID_SHAPE;
    tcm_status s = check_lora_sizes(M, K, R);
    if (s != TCM_OK) return s;
    if (N > kMaxRows || L > kMaxRows) return TCM_ERR_UNSUPPORTED_SHAPE;
    if (M == 1) {  // no step from row to row
        ldx = K;
        ldo = cdiv(N, 4) * 4;
    }
    if (ldx > kMaxLd || ldo > INT32_MAX) return TCM_ERR_UNSUPPORTED_SHAPE;
    if (cdiv(M, 64) * cdiv(N, 64) > INT32_MAX) return TCM_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return TCM_OK;
    const bool adapters = L > 0 && R > 0 && K > 0;
    if (!Out || (K > 0 && (!X || !W)) || (adapters && (!A || !B || !row_adapter || !workspace)))
        return TCM_ERR_NULL_POINTER;
    if (!aligned16(X) || !aligned16(W) || !aligned16(Out) || K % 8 != 0 || ldx % 8 != 0 ||
        (adapters && (!aligned16(A) || !aligned16(B) || !aligned16(workspace) || R % 8 != 0)))
        return TCM_ERR_MISALIGNED;
    LoraArgs a;
    memset(&a, 0, sizeof(a));
    int64_t kpart;
    const int64_t parts = lora_parts(M, K, &kpart);
    if (adapters && workspace_bytes < parts * M * R * 4) return TCM_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    a.X = X;
    a.W = W;
    a.A = A;
    a.B = B;
    a.rows = row_adapter;
    a.ranks = ranks;
    a.scales = scales;
    a.out = Out;
    a.t = (float*)workspace;
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.L = adapters ? (int32_t)L : 0;
    a.R = (int32_t)R;
    a.ldx = (int32_t)ldx;
    a.ldo = (int32_t)ldo;
    a.ksplit = (int32_t)parts;
    a.kpart = (int32_t)kpart;
    return launched(launch_lora(a, (int32_t)dtype, (int32_t)out_dtype, dev.cus, (hipStream_t)stream));
}

tcm_status tcm_qk_norm_rope(const tcm_heads* q, const tcm_heads* k, const tcm_heads* q_out,
                            const tcm_heads* k_out, int64_t T, int64_t Hq, int64_t Hk,
                            const tcm_rope* rope, tcm_dtype dtype, void* stream) {
    tcm_status s = check_rope(rope, dtype, T, Hq, Hk);
    if (s != TCM_OK || T == 0 || Hq + Hk == 0) return s;
    const int64_t D = rope->head_dim;
    if (Hq > 0 && ((s = check_heads(q, T, Hq)) != TCM_OK || (s = check_written(q_out, T, Hq, D)) != TCM_OK)) return s;
    if (Hk > 0 && ((s = check_heads(k, T, Hk)) != TCM_OK || (s = check_written(k_out, T, Hk, D)) != TCM_OK)) return s;
    DeviceInfo dev;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    RopeArgs a;
    fill_rope(&a, rope, T, Hq, Hk);
    if (Hq > 0) a.q = view(q, T, Hq), a.qo = view(q_out, T, Hq);
    if (Hk > 0) a.k = view(k, T, Hk), a.ko = view(k_out, T, Hk);
    return launched(launch_norm_rope(a, (int32_t)dtype, (int32_t)rope->layout, (hipStream_t)stream));
}

tcm_status tcm_qk_norm_rope_cache(const tcm_heads* q, const tcm_heads* k, const tcm_heads* v,
                                  const tcm_heads* q_out, const tcm_cache* cache,
                                  const int32_t* slots, int64_t T, int64_t Hq, int64_t Hk,
                                  const tcm_rope* rope, tcm_dtype dtype, void* stream) {
    tcm_status s = check_rope(rope, dtype, T, Hq, Hk);
    if (s != TCM_OK) return s;
    const int64_t D = rope->head_dim;
    if ((s = check_cache(cache, dtype, Hk, D, true)) != TCM_OK) return s;
    if (T == 0 || Hq + Hk == 0) return TCM_OK;
    if (!slots) return TCM_ERR_NULL_POINTER;
    if (Hq > 0 && ((s = check_heads(q, T, Hq)) != TCM_OK || (s = check_written(q_out, T, Hq, D)) != TCM_OK)) return s;
    if (Hk > 0 && ((s = check_heads(k, T, Hk)) != TCM_OK || (s = check_heads(v, T, Hk)) != TCM_OK)) return s;
    DeviceInfo dev;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    RopeArgs a;
    fill_rope(&a, rope, T, Hq, Hk);
    if (Hq > 0) a.q = view(q, T, Hq), a.qo = view(q_out, T, Hq);
    if (Hk > 0) a.k = view(k, T, Hk), a.v = view(v, T, Hk);
    a.Hv = (int32_t)Hk;
    a.slots = slots;
    a.num_slots = cache->pages * cache->page_size;
    a.page_size = (int32_t)cache->page_size;
    a.page_shift = shift_of(cache->page_size);
    a.cache_e4m3 = cache->dtype == TCM_E4M3;
    const int64_t es = a.cache_e4m3 ? 1 : 2;
    a.kc = cache->k;
    a.vc = cache->v;
    a.k_page = step_bytes(cache->pages, cache->k_page_stride, es);
    a.k_tok = step_bytes(cache->page_size, cache->k_token_stride, es);
    a.k_head = step_bytes(Hk, cache->k_head_stride, es);
    a.v_page = step_bytes(cache->pages, cache->v_page_stride, es);
    a.v_tok = step_bytes(cache->page_size, cache->v_token_stride, es);
    a.v_head = step_bytes(Hk, cache->v_head_stride, es);
    a.k_scale = scale_parts(cache->k_scale);
    a.v_scale = scale_parts(cache->v_scale);
    return launched(launch_norm_rope(a, (int32_t)dtype, (int32_t)rope->layout, (hipStream_t)stream));
}

tcm_status tcm_qk_norm_rope_bwd_workspace(int64_t head_dim, int64_t* bytes) {
    if (!bytes) return TCM_ERR_NULL_POINTER;
    if (head_dim < 1) return TCM_ERR_INVALID_SHAPE;
    if (head_dim > kMaxHeadDim || head_dim % 8 != 0) return TCM_ERR_UNSUPPORTED_SHAPE;
    *bytes = bwd_workspace(head_dim);
    return TCM_OK;
}

tcm_status tcm_qk_norm_rope_bwd(const tcm_heads* dq_out, const tcm_heads* dk_out,
                                const tcm_heads* q, const tcm_heads* k, const tcm_heads* dq,
                                const tcm_heads* dk, float* dq_weight, float* dk_weight, int64_t T,
                                int64_t Hq, int64_t Hk, const tcm_rope* rope, tcm_dtype dtype,
                                void* workspace, int64_t workspace_bytes, void* stream) {
    tcm_status s = check_rope(rope, dtype, T, Hq, Hk);
    if (s != TCM_OK) return s;
    const int64_t D = rope->head_dim;
    const bool any = T > 0 && Hq + Hk > 0, dw = dq_weight || dk_weight;
    // (without the norm there are no weights)
    if (dw && !rope->norm) return TCM_ERR_INVALID_ARGUMENT;
    if (!any && !dw) return TCM_OK;
    for (int i = 0; any && i < 2; ++i) {
        const int64_t H = i ? Hk : Hq;
        if (H == 0) continue;
        if ((s = check_heads(i ? dk_out : dq_out, T, H)) != TCM_OK) return s;
        if (rope->norm && (s = check_heads(i ? k : q, T, H)) != TCM_OK) return s;
        if ((s = check_written(i ? dk : dq, T, H, D)) != TCM_OK) return s;
    }
    if (dw) {
        if (!workspace) return TCM_ERR_NULL_POINTER;
        if (!aligned16(workspace)) return TCM_ERR_MISALIGNED;
        if (workspace_bytes < bwd_workspace(D)) return TCM_ERR_WORKSPACE;
    }
    DeviceInfo dev;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    RopeArgs a;
    fill_rope(&a, rope, any ? T : 0, Hq, Hk);
    if (any && Hq > 0) {
        a.dqo = view(dq_out, T, Hq), a.qo = view(dq, T, Hq);
        if (rope->norm) a.q = view(q, T, Hq);
    }
    if (any && Hk > 0) {
        a.dko = view(dk_out, T, Hk), a.ko = view(dk, T, Hk);
        if (rope->norm) a.k = view(k, T, Hk);
    }
    a.partial = dw ? (float*)workspace : nullptr;
    a.dwq = dq_weight;
    a.dwk = dk_weight;
    return launched(launch_norm_rope_bwd(a, (int32_t)dtype, (int32_t)rope->layout, (hipStream_t)stream));
}

tcm_status tcm_paged_attention_workspace(int64_t B, int64_t Hq, int64_t Hk, int64_t D,
                                         int64_t max_len, int64_t* bytes) {
    if (!bytes) return TCM_ERR_NULL_POINTER;
    tcm_status s = check_attn_sizes(B, Hq, Hk, D, max_len);
    if (s != TCM_OK) return s;
    *bytes = Hk > 0 ? attn_workspace(most_chunks(B, Hq, Hk, max_len), Hq, D) : 0;
    return TCM_OK;
}

tcm_status tcm_paged_attention(const tcm_heads* q, const tcm_cache* cache,
                               const int32_t* block_table, int64_t table_stride,
                               const int32_t* lengths, int64_t max_len, const tcm_heads* out,
                               float* lse, int64_t B, int64_t Hq, int64_t Hk, int64_t D,
                               float scale, int64_t window, tcm_dtype dtype, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    if (!half_type(dtype)) return TCM_ERR_UNSUPPORTED_DTYPE;
    tcm_status s = check_attn_sizes(B, Hq, Hk, D, max_len);
    if (s != TCM_OK) return s;
    if (window < 0 || table_stride < 0) return TCM_ERR_INVALID_SHAPE;
    if (table_stride > INT32_MAX) return TCM_ERR_UNSUPPORTED_SHAPE;
    if ((s = check_cache(cache, dtype, Hk, D, false)) != TCM_OK) return s;
    if (cache->dtype == TCM_E4M3 && D % 16 != 0) return TCM_ERR_MISALIGNED;
    if (B == 0 || Hq == 0) return TCM_OK;
    if (!lengths || (table_stride > 0 && !block_table)) return TCM_ERR_NULL_POINTER;
    if ((s = check_heads(q, B, Hq)) != TCM_OK || (s = check_written(out, B, Hq, D)) != TCM_OK) return s;
    // no page, no key
    if (cache->pages == 0) max_len = 0;
    // the first tile of a window begins up to 31 keys before it
    const int64_t span = window > 0 && window + 31 < max_len ? window + 31 : max_len;
    const Split sp = split_of(B, Hq, Hk, span);
    if (split_units(B, Hq, Hk) > kMostGroups / sp.n) return TCM_ERR_UNSUPPORTED_SHAPE;
    if (sp.n > 1) {
        if (!workspace) return TCM_ERR_NULL_POINTER;
        if (!aligned16(workspace)) return TCM_ERR_MISALIGNED;
        if (workspace_bytes < attn_workspace(B * sp.n, Hq, D)) return TCM_ERR_WORKSPACE;
    }
    DeviceInfo dev;
    if ((s = device_info(&dev)) != TCM_OK) return s;
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    const bool e4m3 = cache->dtype == TCM_E4M3;
    const int64_t es = e4m3 ? 1 : 2;
    a.q = view(q, B, Hq);
    a.out = view(out, B, Hq);
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
    a.lse = lse;
    if (sp.n > 1) {
        a.po = (float*)workspace;
        a.pml = a.po + B * Hq * sp.n * D;
    }
    a.B = (int32_t)B;
    a.Hq = (int32_t)Hq;
    a.Hk = (int32_t)Hk;
    a.G = (int32_t)(Hq / Hk);
    a.D = (int32_t)D;
    a.pages = (int32_t)cache->pages;
    a.page_size = (int32_t)cache->page_size;
    a.page_shift = shift_of(cache->page_size);
    a.max_len = (int32_t)max_len;
    a.window = window > max_len ? 0 : (int32_t)window;
    a.chunk = (int32_t)sp.chunk;
    a.splits = (int32_t)sp.n;
    a.heads = (int32_t)sp.heads;
    a.qblocks = (int32_t)cdiv(Hq / Hk, 16);
    a.scale_log2 = scale * (e4m3 ? cache->k_scale : 1.0f) * 1.4426950408889634f;
    a.v_scale = e4m3 ? cache->v_scale : 1.0f;
    return launched(launch_paged_attention(a, (int32_t)dtype, e4m3, (hipStream_t)stream));
}

}  // extern "C"
