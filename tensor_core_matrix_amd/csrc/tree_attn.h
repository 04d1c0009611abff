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
// barrier; more: 4 x 1 and tiles of 64, one barrier a tile.
//
// The work is dealt evenly: the tiles of all blocks of rows of all heads and sequences are numbered, and every
// workgroup takes a stretch of as many, over the ends of blocks where they come.  (With a chunk of keys a
// workgroup, sequences of different lengths left the device idle for half of the time.)  A block that lies in
// one stretch is written at once; a stretch begins and ends inside a block at most once each, and tree_join_kernel
// joins those parts.  The host sees no length, so each workgroup adds up the tiles of the sequences itself.
//
// Measured on an MI355X, heads of 128, 32 over 8 (E4M3: 64 over 8), lengths drawn evenly up to the one given, bf16,
// by the lengths drawn: 16 trees of 64 tokens, 4096 keys 66 to 77 us (of them 12 in the join), 32 trees of 16 over
// an E4M3 cache of 4096 78 to 87, 5 tokens in a row on 2 x 65537 keys (fp16) 83 to 99, 9 on up to 700 16.
// Long contexts with few rows are bound by memory; with 128 rows the matrix cores are busy for 42 % of the time,
// vector instructions for 51 %, and the two waves of a SIMD wait for LDS, barriers and each other's products for the
// rest: no single part left out (the second part of P, the exponentials, reads from LDS) gains more than 3 us.
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
    int base;        // where the first tile of the sequence begins
    int sure, safe;  // keys [sure, safe) are seen by every row
};
// (starts and lengths of b as they were loaded)
__device__ __forceinline__ TreeRange tree_sequence(const TreeArgs& p, int start, int stop, int length) {
    TreeRange r;
    const int64_t room = p.table_stride * (int64_t)p.page_size;
    int len = min(max(length, 0), p.max_len);
    if (len > room) len = (int)room;
    r.row0 = max(start, 0);
    r.all = max(stop - r.row0, 0);
    r.m = max(min(min(r.all, p.max_nodes), p.T - r.row0), 0);
    r.context = max(len - r.all, 0);
    r.lo = p.window > 0 ? max(0, r.context - p.window + (p.tree ? 0 : 1)) : 0;
    r.end = len;
    r.base = r.lo & ~31;
    return r;
}
__device__ __forceinline__ TreeRange tree_range(const TreeArgs& p, int b, int blk) {
    TreeRange r = tree_sequence(p, scalar_int(p.starts + b), scalar_int(p.starts + b + 1), scalar_int(p.lengths + b));
    const int first = blk * p.rows / p.G, last = min((blk * p.rows + p.rows - 1) / p.G, r.m - 1);
    const bool chain = !p.tree;
    r.safe = chain ? min(r.end, r.context + first + 1) : r.context;
    r.sure = 0;
    if (p.window > 0) {
        // (a token's bits number 0 to `all`)
        if (chain) r.lo = max(0, r.context + first - p.window + 1);
        r.sure = max(0, chain ? r.context + last - p.window + 1 : min(r.context, r.context + r.all - p.window));
    }
    if (chain) r.end = min(r.end, r.context + last + 1);
    return r;
}

// The work in steps: a tile is one, and what a block of rows takes beside its tiles -- finding its keys, its
// first copies and masks, and storing -- kTreeSetup, its first ones.  Stretches of them: `groups`, the first
// `more` one longer than `each`.
struct TreeShare {
    int64_t each;
    int groups, more;
    __device__ __forceinline__ int64_t begin(int w) const { return w * each + min(w, more); }
    __device__ __forceinline__ int owner(int64_t step) const {
        const int64_t longer = more * (each + 1);
        return step < longer ? (int)(step / (each + 1)) : more + (int)((step - longer) / each);
    }
};
// A sequence that has steps: [before, before + cost), `tiles` + kTreeSetup for each block of rows of each head.
struct TreePlace {
    int64_t before, cost;
    int b, blocks, tiles;
};
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)(uint32_t)uniform((int)x) | (int64_t)uniform((int)(x >> 32)) << 32;
}
__device__ __forceinline__ int64_t lanes_before(int64_t x) {  // the sum of x over this lane and those before
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t y = __shfl_up(x, d);
        x += (int)(threadIdx.x & 63) >= d ? y : 0;
    }
    return x;
}
// The steps of 64 sequences, a lane each, `seen` before them (every lane of the wave is active)
struct TreeLanes {
    int64_t cost, sum;  // sum: with this sequence's
    int blocks, tiles;
};
__device__ __forceinline__ TreeLanes tree_lanes(const TreeArgs& p, int b0, int round, int64_t seen) {
    TreeLanes c = {0, 0, 0, 1};
    const int b = b0 + (threadIdx.x & 63);
    if (b < p.B) {
        const TreeRange r = tree_sequence(p, p.starts[b], p.starts[b + 1], p.lengths[b]);
        c.blocks = (r.m * p.G + p.rows - 1) / p.rows;
        c.tiles = max((r.end - r.base + round - 1) / round, 1);
        c.cost = (int64_t)c.blocks * (c.tiles + kTreeSetup) * p.Hk;
    }
    c.sum = seen + lanes_before(c.cost);
    return c;
}
__device__ __forceinline__ TreeShare tree_share(const TreeArgs& p, int round, TreeLanes& lanes) {
    lanes = tree_lanes(p, 0, round, 0);
    int64_t total = uniform(__shfl(lanes.sum, 63));
    for (int b0 = 64; b0 < p.B; b0 += 64) total = uniform(__shfl(tree_lanes(p, b0, round, total).sum, 63));
    TreeShare s;
    s.groups = (int)min(max(total / kTreeLeast, (int64_t)1), (int64_t)p.groups);
    if (s.groups > 8) s.groups &= ~7;
    s.each = total / s.groups;
    s.more = (int)(total - s.each * s.groups);
    return s;
}
// The sequence of a step; lanes: of the first 64
__device__ __forceinline__ TreePlace tree_place(const TreeArgs& p, int round, int64_t step, const TreeLanes& lanes) {
    TreeLanes c = lanes;
    for (int b0 = 0;; b0 += 64) {
        const uint64_t past = __ballot(step < c.sum);
        if (past != 0 || b0 + 64 >= p.B) {
            const int at = past != 0 ? __builtin_ctzll(past) : 63;
            TreePlace r;
            r.b = b0 + at;
            r.cost = uniform(__shfl(c.cost, at));
            r.before = uniform(__shfl(c.sum, at)) - r.cost;
            r.blocks = uniform(__shfl(c.blocks, at));
            r.tiles = uniform(__shfl(c.tiles, at));
            return r;
        }
        c = tree_lanes(p, b0 + 64, round, uniform(__shfl(c.sum, 63)));
    }
}
// The block of rows of a step: those of a head follow each other.
struct TreeUnit {
    int hk, blk;
    int64_t first;  // its first step
};
__device__ __forceinline__ TreeUnit tree_unit(const TreePlace& s, int64_t step) {
    const int64_t x = step - s.before, unit = x / (s.tiles + kTreeSetup);
    TreeUnit u;
    u.first = s.before + unit * (s.tiles + kTreeSetup);
    u.hk = (int)(unit / s.blocks);
    u.blk = (int)(unit - (int64_t)u.hk * s.blocks);
    return u;
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// copy16_to_lds_asm() of a resource that may come out of vector registers (the compiler keeps scalars there that
// have no place, and brings them back right before their use): five wait states between the vector
// instruction that writes a scalar register and a memory instruction that reads it, which the compiler
// does not insert before inline assembly.  It clobbers no memory: a copy fills the stage that nobody reads until
// the next barrier, which does, and other accesses may be moved over it.
__device__ __forceinline__ void copy16_to_lds_far(__amdgpu_buffer_rsrc_t r, void* lds_wave_base, uint32_t voffset) {
    const uint32_t m0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds_wave_base;
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voffset), "s"(r), "{m0}"(m0));
}

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
__global__ __launch_bounds__((TreeShape<DP, E4M3, WR, RB>::WAVES * 64),
                             (DP > 128 || TreeShape<DP, E4M3, WR, RB>::LDS > 72 * 1024 ? 1 : 2))
void tree_kernel(TreeArgs p) {
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
    // ALIGNED, shared stages: whether the page of 16 keys of a stage is one
    __shared__ __attribute__((aligned(16))) uint32_t there_[2][4];
    // shared stages: whether a wave's part of the values holds one that is not finite
    __shared__ __attribute__((aligned(16))) uint32_t strange_[2][4];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wave % WR, wk = wave / WR;
    const int r16 = lane & 15, g4 = lane >> 4;
    constexpr int ROUND = KT * WK;
    TreeLanes lanes;
    const TreeShare share = tree_share(p, ROUND, lanes);
    if ((int)blockIdx.x >= share.groups) {
        if (p.split && threadIdx.x == 0) p.split[blockIdx.x].parts = 0;
        return;
    }
    // (stretches that follow each other, and so read the same keys now and then, on one XCD)
    const int w = share.groups % 8 == 0 ? blockIdx.x % 8 * (share.groups / 8) + blockIdx.x / 8 : blockIdx.x;
    int64_t step = share.begin(w);
    const int64_t stop = share.begin(w + 1);
    if (step >= stop) {  // (nothing to do at all)
        if (p.split && threadIdx.x == 0) p.split[w].parts = 0;
        return;
    }
    TreePlace place = tree_place(p, ROUND, step, lanes);
    for (bool head = true;; head = false) {
        const TreeUnit unit = tree_unit(place, step);
        const int b = place.b, hk = unit.hk, blk = unit.blk;
        // the tiles [tile0, tile1) of the block, of place.tiles
        const int64_t tile_step = unit.first + kTreeSetup, past = unit.first + kTreeSetup + place.tiles;
        const int tile0 = (int)max(step - tile_step, (int64_t)0), tile1 = (int)(min(stop, past) - tile_step);
        if (head && p.split && threadIdx.x == 0) {
            // A block whose first tiles are the stretch's before this one: its parts are this one's to announce.
            TreeSplit s = {0, b, hk, blk};
            if (step > tile_step && share.owner(tile_step) == w - 1) s.parts = share.owner(past - 1) - w + 2;
            p.split[w] = s;
        }
        if (tile1 > 0) {
            const bool part = tile1 - tile0 < place.tiles;
            // this stretch's first or last part of a block
            const int64_t slot = 2 * (int64_t)w + (tile0 == 0);
            const TreeRange rg = tree_range(p, b, blk);
            // the keys [start, end) of it
            const int64_t from = rg.base + (int64_t)tile0 * ROUND;
            const int start = (int)max(from, (int64_t)(rg.base + (rg.lo - rg.base) / ROUND * ROUND));
            const int end = (int)min((int64_t)rg.end, rg.base + (int64_t)tile1 * ROUND);

            // this lane's rows (those past the last are the last, with zeros for q, and not stored)
            const int row0 = blk * S::ROWS + wr * 16 * RB;
            const int rows = rg.m * p.G - row0;  // of this wave and the later ones
            int tok[RB], qhead[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const int row = row0 + min(16 * i + r16, rows - 1);
                tok[i] = row / p.G;
                qhead[i] = hk * p.G + row - tok[i] * p.G;
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
            // A wave's copies of a tile, 2 NH HALF of them.  The memory pipe takes one in 16 cycles and more, and a
            // wave that asks for the next one waits; so those of a whole tile are spread over the products before.
            struct Copies {
                __amdgpu_buffer_rsrc_t rk[NH], rv[NH];
                char* to[NH];
            };
            auto copy = [&](const Copies& c, int i) {
                const int y = i / (2 * HALF), q = i % HALF;
                if (i / HALF % 2 == 0) copy16_to_lds_far(c.rk[y], c.to[y] + q * 1024, koff[q]);
                else copy16_to_lds_far(c.rv[y], c.to[y] + KT * KB + q * 1024, voff[q]);
            };
            // Asks for a tile; false if its copies are left to the caller.
            auto issue = [&](Tile& t, int stage, bool leave, Copies& c) {
                if constexpr (ALIGNED) {
                    const bool whole = t.key0 >= rg.lo && t.key0 + KT <= end;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int k = t.key0 + 32 * n;
                        t.good[n] = whole ? ~0u : bits_from(rg.lo - k) & ~bits_from(end - k);
                    }
#pragma unroll
                    for (int y = 0; y < NH; ++y) {
                        const int h = WR > 1 ? wr : y;
                        const uint32_t found = __builtin_amdgcn_readfirstlane(t.page[y]);
                        const bool is = found < (uint32_t)p.pages;
                        if constexpr (WR > 1) there_[stage][wr] = is ? 0xffffu << (wr & 1) * 16 : 0u;
                        else if (!is) t.good[0] &= h ? 0x0000ffffu : 0xffff0000u;
                        const uint32_t size = is ? kOutOfRange : 0u, page = is ? found : 0;
                        const uint32_t at = t.key0 + 16 * h - t.entry[y] * p.page_size;
                        c.rk[y] = make_rsrc(kh + (page * (uint64_t)p.k_page + at * (uint64_t)p.k_tok), size);
                        c.rv[y] = make_rsrc(vh + (page * (uint64_t)p.v_page + at * (uint64_t)p.v_tok), size);
                        c.to[y] = stages + stage * S::STAGE + h * 16 * KB;
                    }
                    if (whole) {
                        if (leave) return false;
#pragma unroll
                        for (int i = 0; i < 2 * NH * HALF; ++i) copy(c, i);
                    } else {
#pragma unroll
                        for (int y = 0; y < NH; ++y)
#pragma unroll
                            for (int q = 0; q < HALF; ++q) {
                                const int k = t.key0 + 16 * (WR > 1 ? wr : y) + q * KN + kr;
                                const bool in = k >= rg.lo && k < end;
                                copy16_to_lds_far(c.rk[y], c.to[y] + q * 1024, in ? koff[q] : kOutOfRange);
                                copy16_to_lds_far(c.rv[y], c.to[y] + KT * KB + q * 1024, in ? voff[q] : kOutOfRange);
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
                return true;
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
            // LDS, since both have one counter.  Three tiles on their way, which E4M3 leaves room for, gained
            // nothing: 80 us against 78 for 32 trees of 16.)
            const int first = start + KT * wk;
            const int tiles = first < end ? (end - first + ROUND - 1) / ROUND : 0;
            Tile tile = look(first);
            Tile next = look(first + ROUND);

            // Q as the second operand: lane l holds row l % 16 and 8 elements of each step.  Elements of step
            // s: 32 s + 8 g .. + 7; for E4M3 keys, whose 16-byte pieces cover two steps,
            // 64 (s / 2) + 16 g + 8 (s % 2) .. + 7.  A negative scale is q's sign (a scale of 0 the least there is:
            // masked scores are -infinity times it).
            const float scale = fmaxf(fabsf(p.scale_log2), 0x1p-126f);
            x8 qf[RB][STEPS];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const T* row = (const T*)p.q.p + (int64_t)(rg.row0 + tok[i]) * p.q.ts + (int64_t)qhead[i] * p.q.hs;
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int e = E4M3 ? 64 * (s >> 1) + 16 * g4 + 8 * (s & 1) : 32 * s + 8 * g4;
                    qf[i][s] = 16 * i + r16 < rows && e < p.D ? *(const x8*)(row + e) : (x8){};
                }
            }
            Copies copies;
            if (tiles > 0) issue(tile, 0, false, copies);
            // The first key of the context that a row sees (a chain: of all keys)
            int low[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                low[i] = 0;
                if (p.window > 0) {
                    if (p.tree) {
                        const uint32_t* w = p.tree + (int64_t)(rg.row0 + tok[i]) * p.tree_words;
                        int d = 0;
                        for (int x = 0; x < p.tree_words && 32 * x < rg.all; ++x)
                            d += __builtin_popcount(w[x] & ~bits_from(rg.all - 32 * x));
                        low[i] = min(rg.context + d - p.window, rg.context);
                    } else {
                        low[i] = rg.context + tok[i] - p.window + 1;
                    }
                    low[i] = max(low[i], 0);
                }
            }
            // (used here, so that the compiler's wait for q is not in the loop, where it would be one for the
            // copies)
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

            // Which of the keys 32 n .. of a tile row i of this lane sees.  (Lanes' numbers by way of a register
            // that the compiler does not look through: what the rare tiles need is not to be kept over the others.)
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
            // A tile that not every row sees whole: values that are not finite are added to the rows that see their
            // keys (infinities and NaN: a probability, which is positive, would not change them), and become zeros.
            auto set_apart = [&](int stage, const uint32_t* good, int key0) {
                char* const vt = stages + stage * S::STAGE + KT * KB;
                int own_lane = lane;
                asm volatile("" : "+v"(own_lane));
                bool strange = false;
                for (int i = (wr * 64 + own_lane) * 16; i < KT * KB; i += WR * 1024) {
                    const u32x4_t v = *(const u32x4_t*)(vt + i);
#pragma unroll
                    for (int y = 0; y < 4; ++y) strange = strange || not_finite<T, E4M3>(v[y]);
                }
                if constexpr (WR > 1) {  // (a part of the stage a wave, and all of them come by here)
                    strange_[stage][wr] = __any(strange);
                    barrier_lds();
                    const u32x4_t any = *(const u32x4_t*)strange_[stage];
                    strange = any[0] | any[1] | any[2] | any[3];
                }
                if (!__any(strange)) return;
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
            // The scores of a tile; SPREAD: with the copies of the next one among the products.
            auto scores = [&](auto spread, const char* kt, f32x4_t (*s)[2 * NT]) {
                constexpr int QS = E4M3 ? STEPS / 2 : STEPS, GROUPS = QS * 2 * NT, COPIES = 2 * NH * HALF;
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int h = 0; h < 2 * NT; ++h) s[i][h] = (f32x4_t){};
                i32x4_t kf[2][2 * NT];
                auto read = [&](int st) {
#pragma unroll
                    for (int h = 0; h < 2 * NT; ++h)
                        kf[st & 1][h] = *(const i32x4_t*)(kt + (16 * h + r16) * KB + ((4 * st + g4) ^ swz(r16)) * 16);
                };
                read(0);
#pragma unroll
                for (int st = 0; st < QS; ++st) {
                    if (st + 1 < QS) read(st + 1);
#pragma unroll
                    for (int h = 0; h < 2 * NT; ++h) {
                        const i32x4_t w = kf[st & 1][h];
                        if constexpr (E4M3) {
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                u32x4_t u;
                                u[0] = H::from_fp8(w[2 * y], false);
                                u[1] = H::from_fp8(w[2 * y], true);
                                u[2] = H::from_fp8(w[2 * y + 1], false);
                                u[3] = H::from_fp8(w[2 * y + 1], true);
#pragma unroll
                                for (int i = 0; i < RB; ++i) s[i][h] = H::mma(__builtin_bit_cast(x8, u), qf[i][2 * st + y], s[i][h]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < RB; ++i) s[i][h] = H::mma(__builtin_bit_cast(x8, w), qf[i][st], s[i][h]);
                        }
                        if constexpr (decltype(spread)::value) {
                            const int g = st * 2 * NT + h;
#pragma unroll
                            for (int i = 0; i < COPIES; ++i)
                                if (i * GROUPS / COPIES == g) copy(copies, i);
                        }
                    }
                }
            };
            auto products = [&](int stage, bool plain, bool spread, const uint32_t* good, int key0) {
                const char* const kt = stages + stage * S::STAGE;
                const char* const vt = kt + KT * KB;
                float x[RB][8 * NT];
                f32x4_t s[RB][2 * NT];
                if (spread) scores(std::true_type{}, kt, s);
                else scores(std::false_type{}, kt, s);
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
                            for (int j = 0; j < 8; ++j)
                                x[i][8 * n + j] = sees >> ((j < 4 ? 0 : 16) + (j & 3)) & 1 ? x[i][8 * n + j] : kNegInf;
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
                read_values(0, 0);
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
                        // (Where it is 0, infinities in o become NaN.  Held at the least normal number it keeps them, but of
                        // bf16's largest values too.)
                        const float f = mx[i] == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((mx[i] - m2) * scale);
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
                    if (n > 0) read_values(n, 0);
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

            auto compute = [&](int stage, uint32_t* good, int key0, bool spread) {
                if constexpr (ALIGNED && WR > 1) {
                    const u32x4_t is = *(const u32x4_t*)there_[stage];
                    good[0] &= __builtin_amdgcn_readfirstlane(is[0] | is[1]);
                    good[1] &= __builtin_amdgcn_readfirstlane(is[2] | is[3]);
                }
                bool plain = key0 >= rg.sure && key0 + KT <= rg.safe;
#pragma unroll
                for (int n = 0; n < NT; ++n) plain = plain && good[n] == ~0u;
                if (!plain) set_apart(stage, good, key0);
                if (rows > 0) products(stage, plain, spread, good, key0);
            };
            for (int r = 0; r < tiles; ++r) {
                uint32_t good[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) good[n] = tile.good[n];
                settle(r & 1);
                if constexpr (ALIGNED) wait_vmcnt<0>();
                if constexpr (WR > 1) barrier_lds();
                else wave_lds_exchange();
                bool spread = false;
                if (r + 1 < tiles) {
                    spread = !issue(next, (r + 1) & 1, rows > 0, copies);
                    tile = next;
                    next = look(first + (r + 2) * ROUND);
                }
                compute(r & 1, good, first + r * ROUND, spread);
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
                if (part) {
                    const int64_t at = slot * S::ROWS + row - blk * S::ROWS;
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
                    if (d == 0 && p.lse)
                        p.lse[(int64_t)(rg.row0 + t) * p.Hq + h] = m == kNegInf ? kNegInf : 0.6931471805599453f * m + logf(l);
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
                                store(row0 + 16 * i + r16, d, o[i][m] * down, mx[i], sum[i]);
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
        step = past;
        if (step >= stop) return;
        if (step >= place.before + place.cost) place = tree_place(p, ROUND, step, lanes);
        __syncthreads();  // (the stages, and what met in LDS, are free)
    }
}

// Joins the parts of the blocks of rows that lie in more than one stretch, DL lanes a row; with many parts all
// lanes take one row after the other.  (Few parts are loaded without conditions, all at once: a load under one for
// each part made 14.2 us of 13.2.)
template <class T, int DL>
__global__ __launch_bounds__(256) void tree_join_kernel(TreeArgs p) {
    constexpr int RG = 256 / DL;
    __shared__ float wt[kTreeGroups];
    __shared__ float red[2][4];
    __shared__ __attribute__((aligned(16))) float join[RG][DL * 4];
    const TreeSplit unit = p.split[blockIdx.x + 1];
    const int n = unit.parts, w0 = blockIdx.x;
    if (n == 0) return;
    const TreeRange rg = tree_range(p, unit.b, unit.blk);
    const int rows = min(rg.m * p.G - unit.blk * p.rows, p.rows);
    const int c = threadIdx.x, d = c % DL * 4, g = c / DL;
    // part i of row r: in place 2 (w0 + i) + 1 for the first, which ends its stretch, else 2 (w0 + i)
    auto place_of = [&](int i, int r) { return (2 * (int64_t)(w0 + i) + (i == 0)) * p.rows + r; };
    auto store = [&](int r, f32x4_t a, float top, float l) {
        const int row = unit.blk * p.rows + r, t = row / p.G, h = unit.hk * p.G + row - t * p.G;
        const float z = top == kNegInf ? 0.0f : p.v_scale / l;
        T* out = (T*)p.out.p + (int64_t)(rg.row0 + t) * p.out.ts + (int64_t)h * p.out.hs + d;
        store4<T>(out, a[0] * z, a[1] * z, a[2] * z, a[3] * z);
        if (d == 0 && p.lse)
            p.lse[(int64_t)(rg.row0 + t) * p.Hq + h] = top == kNegInf ? kNegInf : 0.6931471805599453f * top + logf(l);
    };
    // N parts at most, all of whose loads are under way together (past the last: the last one's again)
    auto few = [&](auto most) {
        constexpr int N = decltype(most)::value;
        const int r = blockIdx.y * RG + g;
        if (r >= rows || d >= p.D) return;
        float m[N], l[N], top = kNegInf, sum = 0.0f;
        f32x4_t v[N], a = {};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t at = place_of(min(i, n - 1), r);
            m[i] = p.pml[2 * at];
            l[i] = p.pml[2 * at + 1];
            v[i] = *(const f32x4_t*)(p.po + at * p.D + d);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, m[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i >= n || m[i] == kNegInf) continue;
            const float f = __builtin_amdgcn_exp2f(m[i] - top);
            sum += f * l[i];
            a += f * v[i];
        }
        store(r, a, top, sum);
    };
    if (n <= 2) return few(std::integral_constant<int, 2>{});
    if (n <= 4) return few(std::integral_constant<int, 4>{});
    if (n <= 16) return few(std::integral_constant<int, 16>{});
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        float top = kNegInf, l = 0.0f;
        for (int i = c; i < n; i += 256) top = fmaxf(top, p.pml[2 * place_of(i, r)]);
#pragma unroll
        for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
        if ((c & 63) == 0) red[0][c >> 6] = top;
        __syncthreads();
        top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
        for (int i = c; i < n; i += 256) {
            const float m = p.pml[2 * place_of(i, r)];
            const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - top);
            wt[i] = f;
            l += m == kNegInf ? 0.0f : f * p.pml[2 * place_of(i, r) + 1];
        }
#pragma unroll
        for (int x = 1; x < 64; x *= 2) l += __shfl_xor(l, x);
        if ((c & 63) == 0) red[1][c >> 6] = l;
        __syncthreads();
        l = red[1][0] + red[1][1] + red[1][2] + red[1][3];
        f32x4_t a = {};
        if (d < p.D)
#pragma unroll 4
            for (int i = g; i < n; i += RG) a += wt[i] * *(const f32x4_t*)(p.po + place_of(i, r) * p.D + d);
        *(f32x4_t*)&join[g][d] = a;
        __syncthreads();
        if (g == 0 && d < p.D) {
#pragma unroll
            for (int i = 1; i < RG; ++i) a += *(f32x4_t*)&join[i][d];
            store(r, a, top, l);
        }
        __syncthreads();  // (the arrays are free)
    }
}

template <class T, int DP, bool E4M3, bool ALIGNED, int WR, int RB>
hipError_t run_shape(const TreeArgs& a, hipStream_t st) {
    typedef TreeShape<DP, E4M3, WR, RB> S;
    hipLaunchKernelGGL((tree_kernel<T, DP, E4M3, ALIGNED, WR, RB>), dim3(a.groups), dim3(S::WAVES * 64), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.po) return e;
    // Few parts: 256 / (DP / 4) rows a workgroup; many: rows y, y + the grid's, .. one by one.  (32 for blocks of 128
    // rows, half of which go at once where parts are few, took 13.2 us for 512 parts, 16 take 11.9; for blocks of 64
    // rows and 32 parts 16 take 8.4, 32 7.5.)
    constexpr int RG = 256 / (DP / 4), MOST = S::ROWS > 64 ? 16 : 32;
    static_assert(MOST * RG >= S::ROWS, "all rows of a block");
    hipLaunchKernelGGL((tree_join_kernel<T, DP / 4>), dim3(a.groups - 1, min(min(S::ROWS, a.max_nodes * a.G), MOST)), dim3(256),
                       0, st, a);
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
    return a.page_size % 16 == 0 ? run_main<T, DP, E4M3, true>(a, st) : run_main<T, DP, E4M3, false>(a, st);
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
