// Host/device shared definitions of the layer operators (adapters, norm and
// rotation of heads, paged attention); not part of the public ABI.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace tcm {

constexpr int kMaxHeadDim = 256;

// ---- norm and rotation of heads (rope.hip) ----------------------------------

// A view of tokens x heads x D; strides in elements.
struct HeadView {
    void* p;
    int64_t ts, hs;
};

// A scale 2^e m, 1/2 <= |m| < 1, with 1 / m and 448 |m|.
struct E4m3Scale {
    float m, inv, top;
    int32_t e;
};

struct RopeArgs {
    HeadView q, k, v;    // inputs (backward: the inputs of the forward pass)
    HeadView qo, ko;     // outputs (backward: gradients of the inputs)
    HeadView dqo, dko;   // backward: gradients of the outputs
    const int32_t* pos;
    const double* inv_freq;
    const void* wq;
    const void* wk;
    float eps, factor;
    int32_t T, Hq, Hk, Hv;
    int32_t D, rot;
    int32_t norm, w_f32;
    int32_t tb;   // tokens of one workgroup (of one step of it, backward)
    int32_t per;  // (token, head) items of one workgroup of grid.y
    // cache: keys and values go there (slots != NULL)
    const int32_t* slots;
    int64_t num_slots;
    int32_t page_size, cache_e4m3;
    int32_t page_shift;  // log2 of page_size where it is a power of two, else -1
    float inv_d;         // 1 / D
    int64_t k_page, k_tok, k_head, v_page, v_tok, v_head;  // bytes
    void* kc;
    void* vc;
    E4m3Scale k_scale, v_scale;
    // backward: gridDim.x rows of 2 x D partial weight gradients, then their sums
    float* partial;
    float* dwq;
    float* dwk;
};

constexpr int kRopeTrig = 1024;      // (token, pair) angles of one workgroup
constexpr int kRopeTokens = 64;      // tokens of one workgroup, at most
constexpr int kRopeBwdGrid = 1024;   // workgroups of the backward pass

hipError_t launch_norm_rope(const RopeArgs& a, int32_t dtype, int32_t layout, hipStream_t st);
hipError_t launch_norm_rope_bwd(const RopeArgs& a, int32_t dtype, int32_t layout, hipStream_t st);

// ---- attention of one token over a paged cache (paged_attn.hip) ---------------

struct AttnArgs {
    HeadView q, out;
    const char* kc;
    const char* vc;
    int64_t k_page, k_tok, k_head, v_page, v_tok, v_head;  // bytes
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lengths;
    float* lse;
    float* po;   // split: B x Hq x splits x D partial sums,
    float* pml;  // and B x Hq x splits pairs (maximum in base 2, sum)
    int32_t B, Hq, Hk, G, D;
    int32_t pages, page_size;
    int32_t page_shift;  // log2 of page_size where it is a power of two, else -1
    int32_t max_len, window;
    int32_t chunk, splits;
    int32_t heads;    // key-value heads of a workgroup: 1, or 4, one a wave
    int32_t qblocks;  // blocks of 16 query heads of one key-value head
    float scale_log2, v_scale;
};

constexpr int kAttnMaxSplits = 256;

hipError_t launch_paged_attention(const AttnArgs& a, int32_t dtype, bool e4m3, hipStream_t st);

// ---- projection with adapters (lora.hip) ------------------------------------

struct LoraArgs {
    const void* X;
    const void* W;
    const void* A;
    const void* B;
    const int32_t* rows;   // M adapter numbers
    const int32_t* ranks;  // NULL: all R
    const float* scales;   // NULL: ones
    void* out;
    float* t;  // ksplit x M x R: s_a (X A_a^T) in fp32
    int32_t M, N, K, L, R;
    int32_t ldx, ldo;
    int32_t ksplit;  // parts of K in t
    int32_t kpart;   // K values of one part (a multiple of 1024)
};

constexpr int kLoraMaxRank = 128;

hipError_t launch_lora(const LoraArgs& a, int32_t dtype, int32_t out_dtype, int cus, hipStream_t st);

}  // namespace tcm
