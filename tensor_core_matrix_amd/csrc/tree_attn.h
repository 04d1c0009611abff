// Attention of several new tokens per sequence -- a tree of drafts or a chain -- over a paged
// key-value cache.
//
// The rows of a sequence and key-value head are its m tokens times the G query heads that share
// the head, token by token.  As with one token a sequence, rows are the columns of 16-wide products,
//
//   S^T = K Q^T   (16 keys x 16 rows; a lane holds keys 4 g .. 4 g + 3 of row l % 16, g = l / 16)
//   O^T = V^T P^T (16 elements x 16 rows)
//
// and P goes from the first product's output into the second one's input without leaving its
// lane (as two parts of 8 or 11 bits): the 8 inner positions of lane group g there are keys
// 4 g + j of a tile's first 16 and of its second.
//
// Keys and values go from memory straight into one of two LDS stages, a tile ahead, in rows whose
// 16-byte pieces are exchanged so that operand reads meet all banks; values are read transposed.
// Pieces past a head's end, keys past the sequence's, and holes are offsets out of a buffer's
// range: they arrive as zeros.  (Pages whose size 16 does not divide go through registers, since
// a copy has one base address for its keys.)
//
// WR waves share the stages and take 16 RB rows each; WK groups of WR waves take every WK-th tile
// and meet in LDS at the end.  16 rows or fewer: 1 x 4 and tiles of 32 keys, each wave stages of its own and no
// barrier; more: 4 x 1 and tiles of 64, one barrier a tile.  With more than one chunk of keys tree_join_kernel joins
// the parts.
//
// Which keys a row sees is a word of 32 bits a tile, made for tiles that need it: those that reach
// the sequence's own tokens, the window's edge, the end or a hole.  There a value that is not finite
// is kept from the rows that do not see its key (0 times it would be NaN).
#pragma once

#include <type_traits>

#include "attn_device.h"
#include "paged_rows.h"
#include "step_internal.h"
#include "tcm_device.h"

namespace tcm {

namespace {

// What block `blk` of the rows of sequence b has to do.
struct TreeRange {
    int row0;        // first row of q (token starts[b])
    int m;           // tokens with rows of their own: of the sequence's, those below max_nodes and T
    int all;         // the sequence's tokens
    int context;     // keys before them
    int lo, end;     // the keys [lo, end) that any of the block's rows may see
    int base;        // where the first tile begins
    int sure, safe;  // keys [sure, safe) are seen by every row
};
__device__ __forceinline__ TreeRange tree_range(const TreeArgs& p, int b, int blk) {
    TreeRange r;
    const int64_t room = p.table_stride * (int64_t)p.page_size;
    int len = min(max(scalar_int(p.lengths + b), 0), p.max_len);
    if (len > room) len = (int)room;
    r.row0 = max(scalar_int(p.starts + b), 0);
    r.all = max(scalar_int(p.starts + b + 1) - r.row0, 0);
    r.m = max(min(min(r.all, p.max_nodes), p.T - r.row0), 0);
    r.context = max(len - r.all, 0);
    const int first = blk * p.rows / p.G, last = min((blk * p.rows + p.rows - 1) / p.G, r.m - 1);
    const bool chain = !p.tree;
    r.end = chain ? min(len, r.context + last + 1) : len;
    r.safe = chain ? min(len, r.context + first + 1) : r.context;
    r.lo = r.sure = 0;
    if (p.window > 0) {
        // (a token's bits number 0 to `all`)
        r.lo = max(0, chain ? r.context + first - p.window + 1 : r.context - p.window);
        r.sure = max(0, chain ? r.context + last - p.window + 1 : min(r.context, r.context + r.all - p.window));
    }
    r.base = r.lo & ~31;
    return r;
}
// Chunks of it, at most p.splits (the last one takes what is left)
__device__ __forceinline__ int tree_chunks(const TreeArgs& p, const TreeRange& r) {
    return min((int)(((int64_t)max(r.end - r.base, 0) + p.chunk - 1) / p.chunk), p.splits);
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// bits x .. 31 of a word, for any x
__device__ __forceinline__ uint32_t bits_from(int x) { return x <= 0 ? ~0u : x >= 32 ? 0u : ~0u << x; }

template <class T, bool E4M3>
__device__ __forceinline__ bool not_finite(uint32_t w) {
    if constexpr (E4M3) {
        const uint32_t u = (w & 0x7f7f7f7fu) + 0x01010101u;  // 0x7f: NaN
        return (u & 0x80808080u) != 0;
    } else {
        constexpr uint32_t top = std::is_same<T, __bf16>::value ? 0x7f80u : 0x7c00u;
        return (w & top) == top || (w >> 16 & top) == top;
    }
}

// How the waves of a workgroup share the work, and its LDS.
template <int DP, bool E4M3, int WR_, int RB_>
struct TreeShape {
    static constexpr int WR = WR_, RB = RB_;
    static constexpr int ES = E4M3 ? 1 : 2;
    static constexpr int KB = DP * ES;            // bytes of a key
    static constexpr int NT = WR > 1 ? 2 : 1;     // 32 keys of a tile
    static constexpr int KT = 32 * NT;            // keys of a tile
    static constexpr int STAGE = 2 * KT * KB;     // its keys and values
    // groups of waves over the keys; four pairs of stages fit in LDS up to 256 bytes a key
    static constexpr int WK = WR > 1 ? 1 : KB <= 256 ? 4 : 2;
    static constexpr int WAVES = WR * WK;
    static constexpr int ROWS = 16 * WR * RB;     // of a workgroup
    static constexpr int MEET = WK > 1 ? WK * 16 * (DP + 4) * 4 : 0;
    static constexpr int LDS = 2 * WK * STAGE > MEET ? 2 * WK * STAGE : MEET;
};

// DP: D rounded up to 64, 128 or 256.  ALIGNED: page_size is a multiple of 16, so 16 keys from a multiple
// of 16 on lie in one page.
template <class T, int DP, bool E4M3, bool ALIGNED, int WR, int RB>
__global__ __launch_bounds__((TreeShape<DP, E4M3, WR, RB>::WAVES * 64), (TreeShape<DP, E4M3, WR, RB>::LDS > 72 * 1024 ? 1 : 2)) void tree_kernel(TreeArgs p) {
    typedef TreeShape<DP, E4M3, WR, RB> S;
    typedef Half16<T> H;
    typedef typename H::x8 x8;
    constexpr int ES = S::ES, KB = S::KB, WK = S::WK, NT = S::NT, KT = S::KT;
    constexpr int STEPS = DP / 32;     // products of 32 over the head
    constexpr int VE = DP / 16;        // products of 16 elements
    constexpr int KL = KB / 16;        // lanes that copy a key,
    constexpr int KN = 64 / KL;        // keys of one copy,
    constexpr int HALF = 16 / KN;      // and copies of 16 keys (or values)
    // A wave's part of a tile: 16 keys and their values NH times
    constexpr int NH = 2 * NT / WR;
    static_assert(NH * WR == 2 * NT, "a wave's copies");
    __shared__ __attribute__((aligned(1024))) char lds[S::LDS];
    __shared__ float lm_[RB][WK][16], ll_[RB][WK][16];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wave % WR, wk = wave / WR;
    const int r16 = lane & 15, g4 = lane >> 4;
    // Blocks of rows of one sequence and head read the same keys: their numbers are a multiple of 8
    // apart where the heads' and sequences' count allows it, which is the same XCD.  The next chunk is
    // moved on by one, so that the last chunks of all do not meet on one XCD.
    const int units = p.B * p.Hk, per = units * p.blocks;
    const int split = blockIdx.x / per, rest = blockIdx.x - split * per;
    const int blk = rest / units, unit = (rest - blk * units + split) % units;
    const int b = unit / p.Hk, hk = unit - b * p.Hk;
    const TreeRange rg = tree_range(p, b, blk);
    if (blk * S::ROWS >= rg.m * p.G) return;
    const int start = rg.base + split * p.chunk;
    const int end = split + 1 == p.splits ? rg.end : (int)min((int64_t)rg.end, (int64_t)start + p.chunk);
    if (p.splits > 1 && start >= end) return;

    // this lane's rows (those past the last are the last, with zeros for q, and not stored)
    const int row0 = blk * S::ROWS + wr * 16 * RB;
    const int rows = rg.m * p.G - row0;  // of this wave and the later ones
    int tok[RB], head[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int row = row0 + min(16 * i + r16, rows - 1);
        tok[i] = row / p.G;
        head[i] = hk * p.G + row - tok[i] * p.G;
    }

    // ---- keys and values into LDS ---------------------------------------------------
    // A key's 16-byte piece c lies in LDS at c ^ swz(key), so that the 16 keys of an operand read
    // meet different banks; swz goes by the key's number within 16.
    constexpr int SH = KL >= 16 ? 0 : KL == 8 ? 1 : 2;
    auto swz = [](int key) { return (key >> SH) & ((KL < 16 ? KL : 16) - 1); };
    char* const stages = lds + wk * 2 * S::STAGE;  // a stage: KT keys, KT values
    const int kc = lane % KL, kr = lane / KL;
    const int32_t* const trow = p.table + b * p.table_stride;
    const char* const kh = p.kc + hk * p.k_head;
    const char* const vh = p.vc + hk * p.v_head;
    auto page_of = [&](int key) { return (int)((uint64_t)(uint32_t)key * p.page_magic >> p.page_shift); };
    // ALIGNED, shared stages: whether the page of 16 keys of a stage is one
    __shared__ uint32_t there_[2][4];
    struct Tile {
        int key0;
        int page[NH];       // ALIGNED: of the 16 keys that the wave copies; else [0] of key l % KT of lane l
        int entry[NH];      // and their numbers in the table's row
        uint32_t good[NT];  // the keys that can be used at all (ALIGNED, shared stages: but for their pages)
    };
    auto look = [&](int key0) {
        Tile t;
        t.key0 = key0;
        if constexpr (ALIGNED) {
#pragma unroll
            for (int y = 0; y < NH; ++y) {
                const int key = key0 + 16 * (WR > 1 ? wr : y);
                t.entry[y] = page_of(key);
                t.page[y] = key < end ? trow[t.entry[y]] : -1;
            }
        } else {
            const int key = key0 + (lane & (KT - 1));
            t.entry[0] = page_of(key);
            t.page[0] = key >= rg.lo && key < end ? trow[t.entry[0]] : -1;
        }
        return t;
    };
    // ALIGNED: a lane's offsets from the first of 16 keys (16 token strides are less than 2^31 bytes)
    uint32_t koff[HALF], voff[HALF];
#pragma unroll
    for (int q = 0; q < HALF; ++q) {
        const int key = q * KN + kr, piece = kc ^ swz(key);
        const bool in = 16 * piece < p.D * ES;
        koff[q] = in ? key * (uint32_t)p.k_tok + piece * 16 : kOutOfRange;
        voff[q] = in ? key * (uint32_t)p.v_tok + piece * 16 : kOutOfRange;
    }
    u32x4_t held[ALIGNED ? 1 : 2 * NH * HALF];
    auto issue = [&](Tile& t, int stage) {
        char* const to = stages + stage * S::STAGE;
        if constexpr (ALIGNED) {
            const bool whole = t.key0 >= rg.lo && t.key0 + KT <= end;
#pragma unroll
            for (int n = 0; n < NT; ++n) t.good[n] = whole ? ~0u : bits_from(rg.lo - t.key0 - 32 * n) & ~bits_from(end - t.key0 - 32 * n);
#pragma unroll
            for (int y = 0; y < NH; ++y) {
                const int h = WR > 1 ? wr : y;
                const int key = t.key0 + 16 * h;
                const uint32_t found = __builtin_amdgcn_readfirstlane(t.page[y]);
                const bool is = found < (uint32_t)p.pages;
                if constexpr (WR > 1) there_[stage][wr] = is ? 0xffffu << (wr & 1) * 16 : 0u;
                else if (!is) t.good[0] &= h ? 0x0000ffffu : 0xffff0000u;
                const uint32_t size = is ? kOutOfRange : 0u, page = is ? found : 0;
                const uint32_t at = key - t.entry[y] * p.page_size;
                const __amdgpu_buffer_rsrc_t rk = make_rsrc(kh + (page * (uint64_t)p.k_page + at * (uint64_t)p.k_tok), size);
                const __amdgpu_buffer_rsrc_t rv = make_rsrc(vh + (page * (uint64_t)p.v_page + at * (uint64_t)p.v_tok), size);
                char* const dk = to + h * 16 * KB;
                char* const dv = dk + KT * KB;
                if (whole) {
#pragma unroll
                    for (int q = 0; q < HALF; ++q) copy16_to_lds_asm(rk, dk + q * 1024, koff[q]);
#pragma unroll
                    for (int q = 0; q < HALF; ++q) copy16_to_lds_asm(rv, dv + q * 1024, voff[q]);
                } else {
#pragma unroll
                    for (int q = 0; q < HALF; ++q) {
                        const int k = key + q * KN + kr;
                        const bool in = k >= rg.lo && k < end;
                        copy16_to_lds_asm(rk, dk + q * 1024, in ? koff[q] : kOutOfRange);
                        copy16_to_lds_asm(rv, dv + q * 1024, in ? voff[q] : kOutOfRange);
                    }
                }
            }
        } else {
            const bool ok = (uint32_t)t.page[0] < (uint32_t)p.pages;
            if (!ok) t.page[0] = -1;
            const uint64_t all = __ballot(ok);
#pragma unroll
            for (int n = 0; n < NT; ++n) t.good[n] = (uint32_t)(all >> 32 * n);
#pragma unroll
            for (int y = 0; y < NH; ++y)
#pragma unroll
                for (int q = 0; q < HALF; ++q) {
                    const int key = (WR > 1 ? wr : y) * 16 + q * KN + kr, piece = kc ^ swz(key & 15);
                    const int page = __shfl(t.page[0], key), at = t.key0 + key - __shfl(t.entry[0], key) * p.page_size;
                    u32x4_t& k = held[2 * (y * HALF + q)];
                    u32x4_t& v = held[2 * (y * HALF + q) + 1];
                    k = v = (u32x4_t){};
                    if (page >= 0 && 16 * piece < p.D * ES) {
                        k = *(const u32x4_t*)(kh + page * p.k_page + at * p.k_tok + piece * 16);
                        v = *(const u32x4_t*)(vh + page * p.v_page + at * p.v_tok + piece * 16);
                    }
                }
        }
    };
    // what issue() left in registers
    auto settle = [&](int stage) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int y = 0; y < NH; ++y)
#pragma unroll
                for (int q = 0; q < HALF; ++q) {
                    char* const to = stages + stage * S::STAGE + (WR > 1 ? wr : y) * 16 * KB + q * 1024 + lane * 16;
                    *(u32x4_t*)to = held[2 * (y * HALF + q)];
                    *(u32x4_t*)(to + KT * KB) = held[2 * (y * HALF + q) + 1];
                }
        }
    };

    // ---- the tiles of this group of waves ----------------------------------------------
    // Tile r + 1 is asked for while tile r is computed; its pages were looked up a tile before, by loads that
    // the wait for tile r's copies covers.  (A scalar load's wait would be the next one for an operand from
    // LDS, since both have one counter.)
    constexpr int ROUND = KT * WK;
    const int first = start + KT * wk;
    const int tiles = first < end ? (end - first + ROUND - 1) / ROUND : 0;
    Tile tile = look(first);
    if (tiles > 0) issue(tile, 0);
    Tile next = look(first + ROUND);

    // Q as the second operand: lane l holds row l % 16 and 8 elements of each step.  Elements of step
    // s: 32 s + 8 g .. + 7; for E4M3 keys, whose 16-byte pieces cover two steps,
    // 64 (s / 2) + 16 g + 8 (s % 2) .. + 7.  A negative scale is q's sign (a scale of 0 the least there is:
    // masked scores are -infinity times it).
    const float scale = fmaxf(fabsf(p.scale_log2), 0x1p-126f);
    x8 qf[RB][STEPS];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const T* row = (const T*)p.q.p + (int64_t)(rg.row0 + tok[i]) * p.q.ts + (int64_t)head[i] * p.q.hs;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int e = E4M3 ? 64 * (s >> 1) + 16 * g4 + 8 * (s & 1) : 32 * s + 8 * g4;
            qf[i][s] = 16 * i + r16 < rows && e < p.D ? *(const x8*)(row + e) : (x8){};
        }
    }
    // The first key of the context that a row sees (a chain: of all keys)
    int low[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        low[i] = 0;
        if (p.window > 0) {
            if (p.tree) {
                const uint32_t* w = p.tree + (int64_t)(rg.row0 + tok[i]) * p.tree_words;
                int d = 0;
                for (int x = 0; x < p.tree_words && 32 * x < rg.all; ++x) d += __builtin_popcount(w[x] & ~bits_from(rg.all - 32 * x));
                low[i] = min(rg.context + d - p.window, rg.context);
            } else {
                low[i] = rg.context + tok[i] - p.window + 1;
            }
        }
    }
    // (used here, so that the compiler's wait for q is not in the loop, where it would be one for the copies)
    const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            qf[i][s] = __builtin_bit_cast(x8, __builtin_bit_cast(u32x4_t, qf[i][s]) ^ flip);
            asm volatile("" : "+v"(qf[i][s]));
        }

    f32x4_t o[RB][VE];
    float mx[RB], sum[RB];  // the largest score, unscaled, and the sum of exponentials
#pragma unroll
    for (int i = 0; i < RB; ++i) {
#pragma unroll
        for (int m = 0; m < VE; ++m) o[i][m] = (f32x4_t){};
        mx[i] = kNegInf;
        sum[i] = 0.0f;
    }

    // Which of the keys 32 n .. of a tile row i of this lane sees.  (Lanes' numbers by way of a register that the compiler
    // does not look through: what the rare tiles need is not to be kept over the others.)
    auto row_sees = [&](int i, int n, const uint32_t* good, int key0) {
        const int x0 = key0 + 32 * n - rg.context;  // the first key's number among the tokens
        uint32_t bits;
        if (!p.tree) {
            bits = ~bits_from(tok[i] - x0 + 1);
        } else {
            const uint32_t* words = p.tree + (int64_t)(rg.row0 + tok[i]) * p.tree_words;
            const int w = x0 >> 5, sh = x0 & 31;
            const uint32_t w0 = w >= 0 && w < p.tree_words ? words[w] : 0u;
            const uint32_t w1 = w >= -1 && w + 1 < p.tree_words ? words[w + 1] : 0u;
            bits = __builtin_amdgcn_alignbit(w1, w0, sh) | ~bits_from(-x0);
        }
        return bits & good[n] & bits_from(low[i] - key0 - 32 * n);
    };
    // A tile that not every row sees whole: values that are not finite are added to the rows that see their keys
    // (infinities and NaN: a probability, which is positive, would not change them), and become zeros.
    auto set_apart = [&](int stage, const uint32_t* good, int key0) {
        char* const vt = stages + stage * S::STAGE + KT * KB;
        int own_lane = lane;
        asm volatile("" : "+v"(own_lane));
        bool strange = false;
        for (int i = own_lane * 16; i < KT * KB; i += 1024) {
            const u32x4_t v = *(const u32x4_t*)(vt + i);
#pragma unroll
            for (int y = 0; y < 4; ++y) strange = strange || not_finite<T, E4M3>(v[y]);
        }
        if (!__any(strange)) return;  // (the waves that share the stage agree: they look at the same values)
        if (rows > 0)
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t sees = row_sees(i, n, good, key0);
                    for (int k = 0; k < 32; ++k) {
                        const char* row = vt + (32 * n + k) * KB;
#pragma unroll
                        for (int m = 0; m < VE; ++m) {
                            const int d = 16 * m + 4 * (own_lane >> 4);
                            const char* at = row + ((d * ES / 16) ^ swz(k & 15)) * 16 + d * ES % 16;
                            uint32_t u[2];
                            if constexpr (E4M3) {
                                const uint32_t w = *(const uint32_t*)at;
                                u[0] = H::from_fp8(w, false);
                                u[1] = H::from_fp8(w, true);
                            } else {
                                u[0] = *(const uint32_t*)at;
                                u[1] = *(const uint32_t*)(at + 4);
                            }
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float z = (float)__builtin_bit_cast(T, (uint16_t)(u[y >> 1] >> 16 * (y & 1)));
                                o[i][m][y] += (sees >> k & 1) && !(fabsf(z) < __builtin_inff()) ? z : 0.0f;
                            }
                        }
                    }
                }
        if constexpr (WR > 1) barrier_lds();
        else wave_lds_exchange();
        for (int i = (wr * 64 + own_lane) * 4; i < KT * KB; i += WR * 256) {
            uint32_t v = *(const uint32_t*)(vt + i);
            if constexpr (E4M3) {
#pragma unroll
                for (int y = 0; y < 4; ++y) v = (v >> 8 * y & 0x7f) == 0x7f ? v & ~(0xffu << 8 * y) : v;
            } else {
                v = not_finite<T, E4M3>(v & 0xffffu) ? v & 0xffff0000u : v;
                v = not_finite<T, E4M3>(v & 0xffff0000u) ? v & 0xffffu : v;
            }
            *(uint32_t*)(vt + i) = v;
        }
        if constexpr (WR > 1) barrier_lds();
        else wave_lds_exchange();
    };
    auto products = [&](int stage, bool plain, const uint32_t* good, int key0) {
        const char* const kt = stages + stage * S::STAGE;
        const char* const vt = kt + KT * KB;
        float x[RB][8 * NT];
        f32x4_t s[RB][2 * NT];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int h = 0; h < 2 * NT; ++h) s[i][h] = (f32x4_t){};
#pragma unroll
        for (int st = 0; st < STEPS; st += E4M3 ? 2 : 1)
#pragma unroll
            for (int h = 0; h < 2 * NT; ++h) {
                const char* row = kt + (16 * h + r16) * KB;
                const int sw = swz(r16);
                if constexpr (E4M3) {
                    const i32x4_t w4 = *(const i32x4_t*)(row + ((2 * st + g4) ^ sw) * 16);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        u32x4_t u;
                        u[0] = H::from_fp8(w4[2 * y], false);
                        u[1] = H::from_fp8(w4[2 * y], true);
                        u[2] = H::from_fp8(w4[2 * y + 1], false);
                        u[3] = H::from_fp8(w4[2 * y + 1], true);
#pragma unroll
                        for (int i = 0; i < RB; ++i) s[i][h] = H::mma(__builtin_bit_cast(x8, u), qf[i][st + y], s[i][h]);
                    }
                } else {
                    const x8 kf = *(const x8*)(row + ((4 * st + g4) ^ sw) * 16);
#pragma unroll
                    for (int i = 0; i < RB; ++i) s[i][h] = H::mma(kf, qf[i][st], s[i][h]);
                }
            }
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < 8 * NT; ++j) x[i][j] = s[i][j >> 2][j & 3];
        if (!plain) {
            asm volatile("");  // (a branch: as selects it would run for every tile)
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t sees = row_sees(i, n, good, key0) >> 4 * g4;
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i][8 * n + j] = sees >> ((j < 4 ? 0 : 16) + (j & 3)) & 1 ? x[i][8 * n + j] : kNegInf;
                }
        }
        // Values, 16 elements of 8 keys a lane, asked for before the softmax that their products wait for
        constexpr int VG = RB > 1 || VE < 8 ? 4 : 8;  // products whose values are in registers at once
        x8 v[VG];
        auto read_values = [&](int n, int m0) {
#pragma unroll
            for (int y = 0; y < VG; ++y) {
                const int m = m0 + y;
                if constexpr (E4M3) {
                    // 8 rows of 16 bytes, row r from lanes 2 r and 2 r + 1
                    const int r = r16 >> 1, key = (r < 4 ? 0 : 16) + 4 * g4 + (r & 3);
                    const i32x2_t w = lds_read_tr8(vt + (32 * n + key) * KB + (m ^ swz(key & 15)) * 16 + 8 * (r16 & 1));
                    v[y] = __builtin_bit_cast(x8, (u32x4_t){H::from_fp8(w[0], false), H::from_fp8(w[0], true),
                                                            H::from_fp8(w[1], false), H::from_fp8(w[1], true)});
                } else {
                    // twice 4 rows of 16 elements, row r from lanes 4 r .. 4 r + 3
                    const int key = 4 * g4 + (r16 >> 2), c = 2 * m + (r16 >> 1 & 1);
                    const char* at = vt + (32 * n + key) * KB + (c ^ swz(key)) * 16 + 8 * (r16 & 1);
                    union {
                        s16x4_t half[2];
                        x8 all;
                    } u;
                    u.half[0] = lds_read_tr16(at);
                    u.half[1] = lds_read_tr16(at + 16 * KB);
                    v[y] = u.all;
                }
            }
        };
        float top[RB];
        bool higher = false;
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            top[i] = x[i][0];
#pragma unroll
            for (int j = 1; j < 8 * NT; ++j) top[i] = fmaxf(top[i], x[i][j]);
            top[i] = max_over_groups(top[i]);
            higher = higher || top[i] > mx[i];
        }
        if (__any(higher)) {
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const float m2 = fmaxf(mx[i], top[i]);
                // (o may hold infinities: from the least factor on they stay)
                const float f = mx[i] == kNegInf ? 1.0f : fmaxf(__builtin_amdgcn_exp2f((mx[i] - m2) * scale), 0x1p-126f);
                mx[i] = m2;
                sum[i] *= f;
#pragma unroll
                for (int m = 0; m < VE; ++m)
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[i][m][y] *= f;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            read_values(n, 0);
            x8 upper[RB], lower[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const float m0 = mx[i] == kNegInf ? 0.0f : mx[i] * scale;
                u32x4_t pu, pl;
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    float& e0 = x[i][8 * n + j];
                    float& e1 = x[i][8 * n + j + 1];
                    e0 = __builtin_amdgcn_exp2f(fmaf(e0, scale, -m0));
                    e1 = __builtin_amdgcn_exp2f(fmaf(e1, scale, -m0));
                    sum[i] += e0;
                    sum[i] += e1;
                    uint32_t u, l;
                    H::parts(e0, e1, u, l);
                    pu[j / 2] = u;
                    pl[j / 2] = l;
                }
                upper[i] = __builtin_bit_cast(x8, pu);
                lower[i] = __builtin_bit_cast(x8, pl);
            }
#pragma unroll
            for (int m0 = 0; m0 < VE; m0 += VG) {
                if (m0 > 0) read_values(n, m0);
#pragma unroll
                for (int y = 0; y < VG; ++y)
#pragma unroll
                    for (int i = 0; i < RB; ++i) o[i][m0 + y] = H::mma(v[y], upper[i], o[i][m0 + y]);
#pragma unroll
                for (int y = 0; y < VG; ++y)
#pragma unroll
                    for (int i = 0; i < RB; ++i) o[i][m0 + y] = H::mma(v[y], lower[i], o[i][m0 + y]);
            }
        }
    };

    auto compute = [&](int stage, uint32_t* good, int key0) {
        if constexpr (ALIGNED && WR > 1) {
            const u32x4_t is = *(const u32x4_t*)there_[stage];
            good[0] &= __builtin_amdgcn_readfirstlane(is[0] | is[1]);
            good[1] &= __builtin_amdgcn_readfirstlane(is[2] | is[3]);
        }
        bool plain = key0 >= rg.sure && key0 + KT <= rg.safe;
#pragma unroll
        for (int n = 0; n < NT; ++n) plain = plain && good[n] == ~0u;
        if (!plain) set_apart(stage, good, key0);
        if (rows > 0) products(stage, plain, good, key0);
    };
    for (int r = 0; r < tiles; ++r) {
        uint32_t good[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) good[n] = tile.good[n];
        settle(r & 1);
        if constexpr (ALIGNED) wait_vmcnt<0>();
        if constexpr (WR > 1) barrier_lds();
        else wave_lds_exchange();
        if (r + 1 < tiles) {
            issue(next, (r + 1) & 1);
            tile = next;
            next = look(first + (r + 2) * ROUND);
        }
        compute(r & 1, good, first + r * ROUND);
        wave_lds_exchange();
    }

    // ---- sums, and the groups' parts ----------------------------------------------------
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        sum[i] += __shfl_xor(sum[i], 16);
        sum[i] += __shfl_xor(sum[i], 32);
        // a NaN among the scores passed by the maximum: as an infinite one it makes
        // every later factor of this part NaN and of the others 0
        mx[i] = sum[i] != sum[i] ? -kNegInf : mx[i] * scale;
    }
    // 4 elements from d on of a row with maximum m and sum l
    auto store = [&](int row, int d, f32x4_t a, float m, float l) {
        if (p.splits > 1) {
            const int64_t at = (((int64_t)unit * p.blocks) * S::ROWS + row) * p.splits + split;
            *(f32x4_t*)(p.po + at * p.D + d) = a;
            if (d == 0) {
                p.pml[2 * at] = m;
                p.pml[2 * at + 1] = l;
            }
        } else {
            const int t = row / p.G, h = hk * p.G + row - t * p.G;
            const float n = m == kNegInf ? 0.0f : p.v_scale / l;
            T* out = (T*)p.out.p + (int64_t)(rg.row0 + t) * p.out.ts + (int64_t)h * p.out.hs + d;
            store4<T>(out, a[0] * n, a[1] * n, a[2] * n, a[3] * n);
            if (d == 0 && p.lse) p.lse[(int64_t)(rg.row0 + t) * p.Hq + h] = m == kNegInf ? kNegInf : 0.6931471805599453f * m + logf(l);
        }
    };
    if constexpr (WK == 1) {
        // lane l holds elements 16 m + 4 g .. + 3 of row l % 16
        constexpr float down = 1.0f / H::kLift;
#pragma unroll
        for (int i = 0; i < RB; ++i)
            if (16 * i + r16 < rows)
#pragma unroll
                for (int m = 0; m < VE; ++m) {
                    const int d = 16 * m + 4 * g4;
                    if (d < p.D)
                        store(row0 + 16 * i + r16, d, (f32x4_t){o[i][m][0] * down, o[i][m][1] * down, o[i][m][2] * down, o[i][m][3] * down},
                              mx[i], sum[i]);
                }
    } else {
        float (*const lo_)[16][DP + 4] = (float (*)[16][DP + 4])lds;
        auto top = [&](int i, int q) {
            float t = lm_[i][0][q];
#pragma unroll
            for (int w = 1; w < WK; ++w) t = fmaxf(t, lm_[i][w][q]);
            return t;
        };
#pragma unroll
        for (int i = 0; i < RB; ++i)
            if (g4 == 0) {
                lm_[i][wk][r16] = mx[i];
                ll_[i][wk][r16] = sum[i];
            }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            __syncthreads();  // (the rings end here; the last 16 rows' results are read)
            const float f = mx[i] == kNegInf ? 0.0f : 1.0f / H::kLift * __builtin_amdgcn_exp2f(mx[i] - top(i, r16));
#pragma unroll
            for (int m = 0; m < VE; ++m) {
                f32x4_t v = {o[i][m][0] * f, o[i][m][1] * f, o[i][m][2] * f, o[i][m][3] * f};
                if (mx[i] == kNegInf) v = (f32x4_t){};
                *(f32x4_t*)&lo_[wk][r16][16 * m + 4 * g4] = v;
            }
            __syncthreads();
            for (int z = threadIdx.x; z < 16 * (DP / 4); z += WK * 64) {
                const int q = z / (DP / 4), d = z % (DP / 4) * 4;
                if (16 * i + q >= rows || d >= p.D) continue;
                const float tq = top(i, q);
                f32x4_t a = {};
                float l = 0.0f;
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    a += *(f32x4_t*)&lo_[w][q][d];
                    const float mw = lm_[i][w][q];
                    l += mw == kNegInf ? 0.0f : ll_[i][w][q] * __builtin_amdgcn_exp2f(mw - tq);
                }
                store(row0 + 16 * i + q, d, a, tq, l);
            }
        }
    }
}

// Joins the chunks of one row: DL lanes x 4 elements (blockIdx.z picks which), 256 / DL chunks
// at a time, at most kJoinDeep times.  Every load of a part is under way before the weights
// that it waits for are computed.
constexpr int kTreeJoinDeep = 8;
template <class T, int DL>
__global__ __launch_bounds__(256) void tree_join_kernel(TreeArgs p) {
    __shared__ float wt[kTreeMaxSplits];
    __shared__ float red[2][4];
    __shared__ __attribute__((aligned(16))) float join[256 / DL][DL * 4];
    constexpr int PARTS = 256 / DL;
    const int row = blockIdx.x, unit = blockIdx.y;  // of p.max_nodes * p.G rows of each sequence and head
    const int b = unit / p.Hk, hk = unit - b * p.Hk;
    const int blk = row / p.rows;
    const TreeRange rg = tree_range(p, b, blk);
    if (row >= rg.m * p.G) return;
    const int n = tree_chunks(p, rg);
    const int64_t at0 = ((int64_t)unit * p.blocks * p.rows + row) * p.splits;
    const float* ml = p.pml + 2 * at0;
    const int c = threadIdx.x;
    const int dl = (c % DL) * 4, d = blockIdx.z * DL * 4 + dl, part = c / DL;
    const float m = c < n ? ml[2 * c] : kNegInf;
    const float lc = c < n ? ml[2 * c + 1] : 0.0f;
    f32x4_t v[kTreeJoinDeep];
#pragma unroll
    for (int i = 0; i < kTreeJoinDeep; ++i) {
        const int at = part + i * PARTS;
        v[i] = at < n && d < p.D ? *(const f32x4_t*)(p.po + (at0 + at) * p.D + d) : (f32x4_t){};
    }
    float top = m;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
    if ((c & 63) == 0) red[0][c >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - top);
    wt[c] = f;
    float l = m == kNegInf ? 0.0f : f * lc;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) l += __shfl_xor(l, x);
    if ((c & 63) == 0) red[1][c >> 6] = l;
    __syncthreads();
    l = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    f32x4_t a = {};
#pragma unroll
    for (int i = 0; i < kTreeJoinDeep; ++i) {
        const int at = part + i * PARTS;
        if (at < n) a += wt[at] * v[i];
    }
    *(f32x4_t*)&join[part][dl] = a;
    __syncthreads();
    if (part == 0 && d < p.D) {
#pragma unroll
        for (int i = 1; i < PARTS; ++i) a += *(f32x4_t*)&join[i][dl];
        const float z = top == kNegInf ? 0.0f : p.v_scale / l;
        const int t = row / p.G, h = hk * p.G + row - t * p.G;
        T* out = (T*)p.out.p + (int64_t)(rg.row0 + t) * p.out.ts + (int64_t)h * p.out.hs + d;
        store4<T>(out, a[0] * z, a[1] * z, a[2] * z, a[3] * z);
        if (d == 0 && p.lse)
            p.lse[(int64_t)(rg.row0 + t) * p.Hq + h] = top == kNegInf ? kNegInf : 0.6931471805599453f * top + logf(l);
    }
}

// The same for few chunks: DL lanes a row, 256 / DL rows a workgroup, chunk by chunk.
constexpr int kTreeFew = 16;
template <class T, int DL>
__global__ __launch_bounds__(256) void tree_join_few_kernel(TreeArgs p) {
    const int row = blockIdx.x * (256 / DL) + threadIdx.x / DL, unit = blockIdx.y;
    const int b = unit / p.Hk, hk = unit - b * p.Hk, d = threadIdx.x % DL * 4;
    const int blk = min(row / p.rows, p.blocks - 1);
    // (the block's number differs between the lanes, so its range is read by each)
    const TreeRange rg = tree_range(p, b, blk);
    if (row >= rg.m * p.G || d >= p.D) return;
    const int n = tree_chunks(p, rg);
    const int64_t at = ((int64_t)unit * p.blocks * p.rows + row) * p.splits;
    float m[kTreeFew], l[kTreeFew], top = kNegInf, sum = 0.0f;
    f32x4_t v[kTreeFew], a = {};
#pragma unroll
    for (int i = 0; i < kTreeFew; ++i) {
        m[i] = i < n ? p.pml[2 * (at + i)] : kNegInf;
        l[i] = i < n ? p.pml[2 * (at + i) + 1] : 0.0f;
        v[i] = i < n ? *(const f32x4_t*)(p.po + (at + i) * p.D + d) : (f32x4_t){};
        top = fmaxf(top, m[i]);
    }
#pragma unroll
    for (int i = 0; i < kTreeFew; ++i) {
        if (i >= n) continue;
        const float f = m[i] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[i] - top);
        sum += m[i] == kNegInf ? 0.0f : f * l[i];
        a += f * v[i];
    }
    const float z = top == kNegInf ? 0.0f : p.v_scale / sum;
    const int t = row / p.G, h = hk * p.G + row - t * p.G;
    T* out = (T*)p.out.p + (int64_t)(rg.row0 + t) * p.out.ts + (int64_t)h * p.out.hs + d;
    store4<T>(out, a[0] * z, a[1] * z, a[2] * z, a[3] * z);
    if (d == 0 && p.lse)
        p.lse[(int64_t)(rg.row0 + t) * p.Hq + h] = top == kNegInf ? kNegInf : 0.6931471805599453f * top + logf(sum);
}

template <class T, int DP, bool E4M3, bool ALIGNED, int WR, int RB>
hipError_t run_shape(const TreeArgs& a, hipStream_t st) {
    typedef TreeShape<DP, E4M3, WR, RB> S;
    const dim3 grid((uint32_t)a.splits * a.B * a.Hk * a.blocks);
    hipLaunchKernelGGL((tree_kernel<T, DP, E4M3, ALIGNED, WR, RB>), grid, dim3(S::WAVES * 64), 0, st, a);
    return hipGetLastError();
}
template <class T, int DP, bool E4M3, bool ALIGNED>
hipError_t run_main(const TreeArgs& a, hipStream_t st) {
    if (a.rows == 16) return run_shape<T, DP, E4M3, ALIGNED, 1, 1>(a, st);
    if (a.rows == 64) return run_shape<T, DP, E4M3, ALIGNED, 4, 1>(a, st);
    if constexpr (DP < 256) return run_shape<T, DP, E4M3, ALIGNED, 4, 2>(a, st);
    return hipErrorInvalidValue;
}

template <class T, int DP, bool E4M3>
hipError_t run(const TreeArgs& a, hipStream_t st) {
    const hipError_t e = a.page_size % 16 == 0 ? run_main<T, DP, E4M3, true>(a, st) : run_main<T, DP, E4M3, false>(a, st);
    if (e != hipSuccess || a.splits == 1) return e;
    // a whole row a workgroup where that takes its chunks in kTreeJoinDeep turns, else 32 elements
    const dim3 rows(a.max_nodes * a.G, a.B * a.Hk);
    if (a.splits <= kTreeFew)
        hipLaunchKernelGGL((tree_join_few_kernel<T, DP / 4>), dim3((rows.x + 1024 / DP - 1) / (1024 / DP), rows.y), dim3(256), 0, st, a);
    else if (a.splits <= kTreeJoinDeep * (256 / (DP / 4)))
        hipLaunchKernelGGL((tree_join_kernel<T, DP / 4>), rows, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((tree_join_kernel<T, 8>), dim3(rows.x, rows.y, DP / 32), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace

// The launches of one 16-bit type (a translation unit each)
template <class T>
hipError_t launch_tree(const TreeArgs& a, bool e4m3, hipStream_t st) {
    switch (head_instance(a.D)) {
    case 64: return e4m3 ? run<T, 64, true>(a, st) : run<T, 64, false>(a, st);
    case 128: return e4m3 ? run<T, 128, true>(a, st) : run<T, 128, false>(a, st);
    default: return e4m3 ? run<T, 256, true>(a, st) : run<T, 256, false>(a, st);
    }
}

}  // namespace tcm
