// Host/device shared definitions of the operators of a step that drafts (pages and slots,
// residual norm, 4-bit weights, attention of drafted tokens); not part of the public ABI.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "layer_internal.h"

namespace tcm {

// ---- pages and slots (cache_plan.hip) -----------------------------------------

struct PlanArgs {
    int32_t* lengths;
    const int32_t* change;
    int32_t* table;
    int64_t table_stride;
    int32_t* stack;
    int32_t* count;
    int32_t* starts;
    int32_t* slots;      // NULL: not written
    int32_t* positions;  // NULL: not written
    int32_t* missing;    // NULL: not written
    int32_t B, width, pages, page_size, capacity, T;
    int32_t page_shift;  // log2 of page_size where it is a power of two, else -1
};

hipError_t launch_cache_plan(const PlanArgs& a, hipStream_t st);

// ---- residual norm (norm.hip) ----------------------------------------------------

struct NormArgs {
    const void* x;    // backward: the kept sum
    const void* r;    // residual; backward: the kept sum's gradient
    const void* dy;   // backward
    const void* w;
    void* sum;
    void* out;        // backward: dX
    uint8_t* scale;   // E8M0, with 8-bit results
    int64_t ldx, ldr, lds, ldo, lddy;  // elements
    float eps, inv_d;
    int32_t T, D, w_f32;
    float* partial;   // backward: `groups` rows of D partial weight gradients
    float* dw;
    int32_t groups;
};

constexpr int kMaxNormDim = 32768;
constexpr int kNormBwdGroups = 512;

enum NormOut : int32_t { kNormHalf = 0, kNormF32 = 1, kNormMx = 2 };

hipError_t launch_add_rms_norm(const NormArgs& a, int32_t dtype, NormOut out, hipStream_t st);
hipError_t launch_add_rms_norm_bwd(const NormArgs& a, int32_t dtype, hipStream_t st);

// ---- 4-bit weights (gemm_w4.hip) ---------------------------------------------------

struct W4Args {
    const void* x;
    const uint8_t* w;
    const void* scales;
    const uint8_t* zeros;  // NULL: 8
    void* out;
    int64_t ldo;
    int32_t M, N, K, ldx;
    int32_t gchunks;  // chunks of 32 values of a group
    int32_t gshift;   // log2 of it where it is a power of two, else -1
    int32_t groups;   // groups of a row
    // set by the launch: rows of a workgroup, its waves side by side, and the values of a row of X in LDS at once
    int32_t rows, wn, kc;
};

hipError_t launch_gemm_w4(const W4Args& a, int32_t dtype, bool e2m1, bool out_f32, int cus, hipStream_t st);

// ---- attention of drafted tokens (tree_attn.h, tree_attn_{bf16,f16}.hip) ------------------------------------

// A block of rows whose tiles lie in `parts` stretches, the first one that of the workgroup before (0: none).
struct TreeSplit {
    int32_t parts, b, hk, blk;
};

struct TreeArgs {
    HeadView q, out;
    const char* kc;
    const char* vc;
    int64_t k_page, k_tok, k_head, v_page, v_tok, v_head;  // bytes
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lengths;
    const int32_t* starts;
    const uint32_t* tree;  // NULL: a chain; else tree_words words a token
    int32_t tree_words;    // of 32 bits
    float* lse;
    float* po;   // 2 groups x rows x D partial sums of the blocks that lie in more than one stretch (NULL: none can),
    float* pml;  // and as many pairs (maximum in base 2, sum),
    TreeSplit* split;  // and what each stretch goes on with
    int32_t T, B, Hq, Hk, G, D;
    int32_t pages, page_size;
    uint32_t page_magic;  // n / page_size = n * page_magic >> page_shift for n < 2^31
    int32_t page_shift;
    int32_t max_len, max_nodes, window;
    int32_t groups;  // workgroups, which share the tiles evenly
    int32_t rows;    // of a block of one sequence's rows of a key-value head: 16, 64 or 128
    float scale_log2, v_scale;
};

constexpr int kTreeGroups = 512;   // workgroups at most: two for each of 256 compute units
constexpr int kTreeSetup = 3;      // what a block of rows takes beside its tiles, in tiles
constexpr int kTreeLeast = 2;      // steps of a workgroup at least
// Keys of a tile, the unit that is shared out (of all waves' tiles of 32 where waves have their own)
constexpr int tree_round(int64_t rows, int64_t D, int64_t es) {
    return rows > 16 ? 64 : 32 * ((D <= 64 ? 64 : D <= 128 ? 128 : 256) * es <= 256 ? 4 : 2);
}

hipError_t launch_tree_attention_bf16(const TreeArgs& a, bool e4m3, hipStream_t st);
hipError_t launch_tree_attention_f16(const TreeArgs& a, bool e4m3, hipStream_t st);

}  // namespace tcm
