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
// Keys and values go from memory straight into a ring of LDS stages of 32 keys, in rows whose
// 16-byte pieces are exchanged so that operand reads meet all banks; values are read transposed.
// Pieces past a head's end, keys past the sequence's, and holes are offsets out of a buffer's
// range: they arrive as zeros.  (Pages whose size 16 does not divide go through registers, since
// a copy has one base address for its keys.)
//
// WR waves share a stage and take 16 RB rows each; WK groups of WR waves take every WK-th tile
// and meet in LDS at the end.  16 rows or fewer: 1 x 4, each wave a ring of its own and no
// barrier; more: 4 x 1, one barrier a tile.  With more than one chunk of keys tree_join_kernel joins
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
    static constexpr int TILE = 2 * 32 * KB;      // of 32 keys and values
    // groups of waves over the keys; four rings of two stages fit in LDS up to 256 bytes a key
    static constexpr int WK = WR > 1 ? 1 : KB <= 256 ? 4 : 2;
    static constexpr int NS = WR > 1 ? 3 : 2;     // stages of a ring
    static constexpr int WAVES = WR * WK;
    static constexpr int ROWS = 16 * WR * RB;     // of a workgroup
    static constexpr int RING = WK * NS * TILE;
    static constexpr int MEET = WK > 1 ? WK * 16 * (DP + 4) * 4 : 0;
    static constexpr int LDS = RING > MEET ? RING : MEET;
};

// DP: D rounded up to 64, 128 or 256.  ALIGNED: page_size is a multiple of 16, so the 16 keys of a
// half tile lie in one page.
template <class T, int DP, bool E4M3, bool ALIGNED, int WR, int RB>
__global__ __launch_bounds__((TreeShape<DP, E4M3, WR, RB>::WAVES * 64), (TreeShape<DP, E4M3, WR, RB>::LDS > 72 * 1024 ? 1 : 2)) void tree_kernel(TreeArgs p) {
    typedef TreeShape<DP, E4M3, WR, RB> S;
    typedef Half16<T> H;
    typedef typename H::x8 x8;
    constexpr int ES = S::ES, KB = S::KB, WK = S::WK, NS = S::NS;
    constexpr int STEPS = DP / 32;     // products of 32 over the head
    constexpr int VE = DP / 16;        // products of 16 elements
    constexpr int KL = KB / 16;        // lanes that copy a key,
    constexpr int KN = 64 / KL;        // keys of one copy,
    constexpr int KI = 32 / KN;        // and copies of a tile's keys (and of its values)
    constexpr int NL = 2 * KI / WR;    // a wave's part of both
    __shared__ __attribute__((aligned(1024))) char lds[S::LDS];
    __shared__ float pr_[S::WAVES][32][16];
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
    // Q as the second operand: lane l holds row l % 16 and 8 elements of each step.  Elements of step
    // s: 32 s + 8 g .. + 7; for E4M3 keys, whose 16-byte pieces cover two steps,
    // 64 (s / 2) + 16 g + 8 (s % 2) .. + 7.
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

    // ---- keys and values into LDS ---------------------------------------------------
    // A key's 16-byte piece c lies in LDS at c ^ swz(key), so that the 16 keys of an operand read
    // meet different banks; swz goes by the key's number within 16.
    constexpr int SH = KL >= 16 ? 0 : KL == 8 ? 1 : 2;
    auto swz = [](int key) { return (key >> SH) & ((KL < 16 ? KL : 16) - 1); };
    char* const ring = lds + wk * NS * S::TILE;  // a stage: 32 keys, 32 values
    const int kc = lane % KL, kr = lane / KL;
    const int32_t* const trow = p.table + b * p.table_stride;
    const char* const kh = p.kc + hk * p.k_head;
    const char* const vh = p.vc + hk * p.v_head;
    auto page_of = [&](int key, int& at) {
        const int i = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
        at = key - i * p.page_size;
        return i;
    };
    // Copy q of a wave (0 .. NL - 1): with shared stages, half of the waves copy keys and half
    // values.
    auto is_value = [&](int q) { return WR > 1 ? wr >= WR / 2 : q >= KI; };
    auto piece_of = [&](int q) { return WR > 1 ? (wr % (WR / 2)) * NL + q : q % KI; };
    struct Tile {  // its pages (ALIGNED: of each half; else of key l % 32 of lane l), and its keys
        int page[2], at[2];
        int key0;
        uint32_t good;  // the keys that can be used at all
    };
    auto look = [&](int key0) {
        Tile t;
        t.key0 = key0;
        if constexpr (ALIGNED) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = key0 + 16 * h;
                const int i = page_of(key, t.at[h]);
                t.page[h] = key < end ? scalar_int(trow + i) : -1;
            }
        } else {
            const int key = key0 + (lane & 31);
            const int i = page_of(key, t.at[0]);
            t.page[0] = key >= rg.lo && key < end ? trow[i] : -1;
        }
        return t;
    };
    // ALIGNED: a lane's offsets from the first of 16 keys (16 token strides are less than 2^31 bytes)
    uint32_t voff[ALIGNED ? (WR > 1 ? NL : 2 * (16 / KN > 0 ? 16 / KN : 1)) : 1];
    if constexpr (ALIGNED) {
#pragma unroll
        for (int q = 0; q < (int)(sizeof(voff) / 4); ++q) {
            // (WR == 1: of a half's keys, then of its values)
            constexpr int HALF = 16 / KN;
            const bool val = WR > 1 ? is_value(0) : q >= HALF;
            const int key = (WR > 1 ? piece_of(q) % HALF : q % HALF) * KN + kr;
            const int piece = kc ^ swz(key);
            voff[q] = 16 * piece < p.D * ES ? key * (uint32_t)(val ? p.v_tok : p.k_tok) + piece * 16 : kOutOfRange;
        }
    }
    u32x4_t held[ALIGNED ? 1 : NL];
    auto issue = [&](Tile& t, int stage) {
        char* const to = ring + stage * S::TILE;
        if constexpr (ALIGNED) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if ((uint32_t)t.page[h] >= (uint32_t)p.pages) t.page[h] = -1;
            t.good = ((t.page[0] >= 0 ? 0xffffu : 0u) | (t.page[1] >= 0 ? 0xffff0000u : 0u)) & bits_from(rg.lo - t.key0) &
                     ~bits_from(end - t.key0);
            const bool whole = t.key0 >= rg.lo && t.key0 + 32 <= end;
            constexpr int HALF = 16 / KN;
            __amdgpu_buffer_rsrc_t rk[2], rv[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t size = t.page[h] >= 0 ? kOutOfRange : 0u;
                const int64_t pg = max(t.page[h], 0);
                rk[h] = make_rsrc(kh + pg * p.k_page + t.at[h] * p.k_tok, size);
                rv[h] = make_rsrc(vh + pg * p.v_page + t.at[h] * p.v_tok, size);
            }
#pragma unroll
            for (int q = 0; q < NL; ++q) {
                const int i = piece_of(q);
                uint32_t off;
                if constexpr (WR > 1) off = voff[q];
                else off = voff[(q >= KI ? HALF : 0) + q % HALF];
                if (!whole) {
                    const int key = t.key0 + i * KN + kr;
                    off = key >= rg.lo && key < end ? off : kOutOfRange;
                }
                char* const dst = to + (is_value(q) ? 32 * KB : 0) + i * 1024;
                // (the half is known to the compiler or, with shared stages, to the wave)
                const bool second = i >= KI / 2;
                if (is_value(q)) copy16_to_lds_asm(second ? rv[1] : rv[0], dst, off);
                else copy16_to_lds_asm(second ? rk[1] : rk[0], dst, off);
            }
        } else {
            const bool ok = (uint32_t)t.page[0] < (uint32_t)p.pages;
            if (!ok) t.page[0] = -1;
            t.good = (uint32_t)__ballot(ok);
#pragma unroll
            for (int q = 0; q < NL; ++q) {
                const int key = piece_of(q) * KN + kr, piece = kc ^ swz(key);
                const int page = __shfl(t.page[0], key), at = __shfl(t.at[0], key);
                const char* row = is_value(q) ? vh + max(page, 0) * p.v_page + at * p.v_tok
                                              : kh + max(page, 0) * p.k_page + at * p.k_tok;
                held[q] = (u32x4_t){};
                if (page >= 0 && 16 * piece < p.D * ES) held[q] = *(const u32x4_t*)(row + piece * 16);
            }
        }
    };
    // what issue() left in registers
    auto settle = [&](int stage) {
        if constexpr (!ALIGNED) {
            char* const to = ring + stage * S::TILE;
#pragma unroll
            for (int q = 0; q < NL; ++q)
                *(u32x4_t*)(to + (is_value(q) ? 32 * KB : 0) + piece_of(q) * 1024 + lane * 16) = held[q];
        }
    };

    f32x4_t o[RB][VE];
    float mx[RB], sum[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
#pragma unroll
        for (int m = 0; m < VE; ++m) o[i][m] = (f32x4_t){};
        mx[i] = kNegInf;
        sum[i] = 0.0f;
    }

    auto compute = [&](const char* at, uint32_t good, int key0) {
        const char* const kt = at;
        const char* const vt = at + 32 * KB;
        const bool plain = good == ~0u && key0 >= rg.sure && key0 + 32 <= rg.safe;
        f32x4_t s[RB][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < RB; ++i) s[i][h] = (f32x4_t){};
            const char* row = kt + (16 * h + r16) * KB;
            const int sw = swz(r16);
            if constexpr (E4M3) {
#pragma unroll
                for (int st = 0; st < STEPS; st += 2) {
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
                }
            } else {
#pragma unroll
                for (int st = 0; st < STEPS; ++st) {
                    const x8 kf = *(const x8*)(row + ((4 * st + g4) ^ sw) * 16);
#pragma unroll
                    for (int i = 0; i < RB; ++i) s[i][h] = H::mma(kf, qf[i][st], s[i][h]);
                }
            }
        }
        float x[RB][8];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = s[i][j >> 2][j & 3] * p.scale_log2;
        // the keys of inner positions 0..7 of this lane in the second product
        auto vkey = [&](int j) { return (j < 4 ? 0 : 16) + 4 * g4 + (j & 3); };
        uint32_t seen[RB];
        bool strange = false;  // a value that is not finite
        if (!plain) {
            asm volatile("");  // (a branch: as selects it would run for every tile)
            const int x0 = key0 - rg.context;  // the number of key0 among the tokens
#pragma unroll
            for (int i = 0; i < RB; ++i) {
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
                seen[i] = bits & good & bits_from(low[i] - key0);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = seen[i] >> vkey(j) & 1 ? x[i][j] : kNegInf;
            }
            for (int i = lane * 16; i < 32 * KB; i += 1024) {
                const u32x4_t v = *(const u32x4_t*)(vt + i);
#pragma unroll
                for (int y = 0; y < 4; ++y) strange = strange || not_finite<T, E4M3>(v[y]);
            }
            strange = __any(strange);
        }
        x8 upper[RB], lower[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            float top = x[i][0];
#pragma unroll
            for (int j = 1; j < 8; ++j) top = fmaxf(top, x[i][j]);
            top = max_over_groups(top);
            if (__any(top > mx[i])) {
                const float m2 = fmaxf(mx[i], top);
                const float f = m2 == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(mx[i] - m2);
                mx[i] = m2;
                sum[i] *= f;
#pragma unroll
                for (int m = 0; m < VE; ++m)
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[i][m][y] *= f;
            }
            const float m0 = mx[i] == kNegInf ? 0.0f : mx[i];
            u32x4_t pu, pl;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                x[i][j] = __builtin_amdgcn_exp2f(x[i][j] - m0);
                x[i][j + 1] = __builtin_amdgcn_exp2f(x[i][j + 1] - m0);
                sum[i] += x[i][j];
                sum[i] += x[i][j + 1];
                uint32_t u, l;
                H::parts(x[i][j], x[i][j + 1], u, l);
                pu[j / 2] = u;
                pl[j / 2] = l;
            }
            upper[i] = __builtin_bit_cast(x8, pu);
            lower[i] = __builtin_bit_cast(x8, pl);
        }
        if (!strange) {
#pragma unroll
            for (int m = 0; m < VE; ++m) {
                x8 v;
                if constexpr (E4M3) {
                    // 8 rows of 16 bytes, row r from lanes 2 r and 2 r + 1
                    const int r = r16 >> 1, key = (r < 4 ? 0 : 16) + 4 * g4 + (r & 3);
                    const i32x2_t w = lds_read_tr8(vt + key * KB + (m ^ swz(key & 15)) * 16 + 8 * (r16 & 1));
                    v = __builtin_bit_cast(x8, (u32x4_t){H::from_fp8(w[0], false), H::from_fp8(w[0], true),
                                                         H::from_fp8(w[1], false), H::from_fp8(w[1], true)});
                } else {
                    // twice 4 rows of 16 elements, row r from lanes 4 r .. 4 r + 3
                    const int key = 4 * g4 + (r16 >> 2), c = 2 * m + (r16 >> 1 & 1);
                    const char* at = vt + key * KB + (c ^ swz(key)) * 16 + 8 * (r16 & 1);
                    union {
                        s16x4_t half[2];
                        x8 all;
                    } u;
                    u.half[0] = lds_read_tr16(at);
                    u.half[1] = lds_read_tr16(at + 16 * KB);
                    v = u.all;
                }
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    o[i][m] = H::mma(v, upper[i], o[i][m]);
                    o[i][m] = H::mma(v, lower[i], o[i][m]);
                }
            }
        } else {
            // key by key, and only for the rows that see it
            float (*const pr)[16] = pr_[wave];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                wave_lds_exchange();
#pragma unroll
                for (int j = 0; j < 8; ++j) pr[vkey(j)][r16] = x[i][j] * H::kLift;
                wave_lds_exchange();
                for (int k = 0; k < 32; ++k) {
                    const float f = pr[k][r16];
                    const bool sees = seen[i] >> k & 1;
#pragma unroll
                    for (int m = 0; m < VE; ++m) {
                        const int d = 16 * m + 4 * g4;
                        const char* at = vt + k * KB + ((d * ES / 16) ^ swz(k & 15)) * 16 + d * ES % 16;
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
                            const float v = (float)__builtin_bit_cast(T, (uint16_t)(u[y >> 1] >> 16 * (y & 1)));
                            o[i][m][y] += sees ? f * v : 0.0f;
                        }
                    }
                }
            }
            wave_lds_exchange();
        }
    };

    // ---- the tiles of this group of waves ----------------------------------------------
    constexpr int ROUND = 32 * WK;
    const int first = start + 32 * wk;
    const int tiles = first < end ? (end - first + ROUND - 1) / ROUND : 0;
    if constexpr (ALIGNED) {
        // Tile r + NS - 1 is asked for while tile r is computed; its pages were looked up a tile before
        // (their wait is the scalar loads', apart from the copies').
        uint32_t good[NS] = {};
        Tile t = look(first);
#pragma unroll
        for (int i = 0; i < NS - 1; ++i)
            if (i < tiles) {
                issue(t, i);
                good[i] = t.good;
                t = look(first + (i + 1) * ROUND);
            }
        int stage = 0;
        for (int r = 0; r < tiles; ++r) {
            if (NS > 2 && r + 1 < tiles) wait_vmcnt<(NS - 2) * NL>();
            else wait_vmcnt<0>();
            if constexpr (WR > 1) barrier_lds();
            const int next = stage >= 1 ? stage - 1 : NS - 1;
            if (r + NS - 1 < tiles) {
                issue(t, next);
                good[NS - 1] = t.good;
                t = look(first + (r + NS) * ROUND);
            }
            if (rows > 0) compute(ring + stage * S::TILE, good[0], first + r * ROUND);
#pragma unroll
            for (int i = 0; i + 1 < NS; ++i) good[i] = good[i + 1];
            stage = stage + 1 < NS ? stage + 1 : 0;
        }
    } else if (tiles > 0) {
        Tile t = look(first);
        issue(t, 0);
        int stage = 0;
        for (int r = 0; r < tiles; ++r) {
            const uint32_t good = t.good;
            settle(stage);
            t = look(first + (r + 1) * ROUND);
            if constexpr (WR > 1) barrier_lds();
            else wave_lds_exchange();
            if (r + 1 < tiles) issue(t, 0);
            if (rows > 0) compute(ring + stage * S::TILE, good, first + r * ROUND);
            wave_lds_exchange();
            stage = stage + 1 < NS ? stage + 1 : 0;
        }
    }

    // ---- sums, and the groups' parts ----------------------------------------------------
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        sum[i] += __shfl_xor(sum[i], 16);
        sum[i] += __shfl_xor(sum[i], 32);
        // a NaN among the scores passed by the maximum: as an infinite one it makes
        // every later factor of this part NaN and of the others 0
        if (sum[i] != sum[i]) mx[i] = -kNegInf;
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
    if (a.splits <= kTreeJoinDeep * (256 / (DP / 4)))
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
