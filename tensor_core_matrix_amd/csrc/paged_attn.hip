// Attention of one new token per sequence over a paged key-value cache.
//
// Bound by memory: every key and value of a sequence is read once, whatever the
// number of query heads that share it.  The G query heads of a key-value head
// are the columns of 16-wide matrix products, so that the arithmetic stays far
// below the time of the reads:
//
//   S^T = K Q^T   (16 keys x 16 heads; a lane holds keys 4 g .. 4 g + 3 of head
//                  l % 16, g = l / 16)
//   O^T = V^T P^T (16 elements x 16 heads)
//
// The order of a product's inner index is free as long as both operands share
// it.  So the 8 inner positions of lane group g in the second product are the
// keys whose scores the lane already holds -- 4 g + j of a tile's first 16 keys
// and of its second -- and P goes from one product's output into the next one's
// input without leaving its lane.  V is read 8 keys x D / 16 elements a lane
// (lane c = l % 16 takes elements c D / 16 .. of each of its 8 keys, so 16 lanes
// read a whole row), and turned into the 8-keys-of-one-element form by byte
// permutations within the lane.  A probability is cut to the type's 8 or 11 bits
// there, and what that leaves is rounded and multiplied too: 16 or 22 bits together, so
// that the result's error is its own rounding (one product in bf16: a third more).  The
// second products cost up to 1.5 % (64 sequences of up to 4096 keys 101.6 us, and 101.1
// without; 32 of up to 8192 in E4M3 68.0 and 67.0), 1 to 3 with heads above 128.
// Maximum and sum of a head's softmax live in its lanes too.  K is read in whole rows
// and goes through the wave's own LDS area: read in the operand's pattern of 16 rows x
// 64 bytes, memory gives 5.2 TB/s to a kernel that does nothing else, in whole rows
// 6.4.  Nothing waits for another wave until a workgroup's four join at the end.
//
// A workgroup takes a chunk of a sequence's keys, for one key-value head with its
// tiles dealt to the four waves or for four heads, one a wave; the next tile's
// keys and values are on their way while one is computed.  With more than one
// chunk the partial results go to the workspace and attn_join_kernel joins them.
//
// Bound by reads: one sequence of 131001 keys (32 query, 8 key-value heads of 128,
// fp16) takes 86 us, 6.3 TB/s, and 5 for the join; 64 sequences of up to 4096 keys
// 98 us, 5.6 TB/s; 32 of up to 8192 in E4M3 63 us, 4.8 TB/s; 200 keys 8.1 us.
#include <type_traits>

#include "attn_device.h"
#include "layer_internal.h"
#include "paged_rows.h"
#include "tcm_device.h"

namespace tcm {

namespace {

// The keys [lo, len) of sequence b, and where the first tile begins.
struct Range {
    int base, lo, len;
};
__device__ __forceinline__ Range range_of(const AttnArgs& p, int b) {
    Range r;
    const int64_t room = p.table_stride * (int64_t)p.page_size;
    int len = scalar_int(p.lengths + b);
    len = len < 0 ? 0 : len;
    len = min(len, p.max_len);
    if (len > room) len = (int)room;
    r.len = len;
    r.lo = p.window > 0 && len > p.window ? len - p.window : 0;
    r.base = r.lo & ~31;
    return r;
}

// DP: D rounded up to 64, 128 or 256.  E4M3: the cache's elements are E4M3
// bytes.  ALIGNED: page_size is a multiple of 16, so the 16 keys of a half
// tile lie in one page, whose number is looked up once.
template <class T, int DP, bool E4M3, bool ALIGNED>
__global__ __launch_bounds__(256, DP == 256 ? 1 : DP == 128 && E4M3 && ALIGNED ? 3 : 2) void attn_kernel(AttnArgs p) {
    typedef Half16<T> H;
    typedef typename H::x8 x8;
    constexpr int ES = E4M3 ? 1 : 2;
    constexpr int STEPS = DP / 32;          // products of 32 over the head
    constexpr int VE = DP / 16;             // elements of a value row a lane holds
    constexpr int VW = VE * ES / 4;         // words of a lane's piece of a value row,
    constexpr int VB = value_load(DP, ES);  // bytes of one load of it
    constexpr int VL = VW * 4 / VB;         // and its loads
    constexpr int KB = DP * ES;             // bytes of a key
    constexpr int KL = KB / 16;             // lanes that read a key,
    constexpr int KN = 64 / KL;             // keys of one read
    constexpr int KI = 32 / KN;             // and reads of a tile
    // the tile's keys, one area a wave; at the end the waves' results
    constexpr int OB = 4 * 16 * (DP + 4) * 4, KA = 32 * KB;
    __shared__ __attribute__((aligned(1024))) char lds[OB > 4 * KA ? OB : 4 * KA];
    float (*const lo_)[16][DP + 4] = (float (*)[16][DP + 4])lds;
    __shared__ float lm_[4][16], ll_[4][16];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    // Chunk by chunk over all sequences and key-value heads.  Workgroups are dealt
    // to the 8 XCDs in turn, so a sequence's next chunk is moved on by one: were
    // the chunk's number the XCD's (or the sequence's, for a count of sequences
    // that 8 divides), the XCD of the last chunks would idle.
    const int groups = p.Hk / p.heads;  // of key-value heads
    const int units = p.B * groups, per = units * p.qblocks;
    const int split = blockIdx.x / per, rest = blockIdx.x - split * per;
    const int qb = rest / units, unit = (rest - qb * units + split) % units;
    const int b = unit / groups, hw = wave & (p.heads - 1), kw = wave / p.heads;
    const int hk = (unit - b * groups) * p.heads + hw;
    const int round = 128 / p.heads;  // keys of a round of the workgroup's waves
    const int h0 = hk * p.G + qb * 16, nh = min(16, p.G - qb * 16);
    const Range rg = range_of(p, b);
    const int start = rg.base + split * p.chunk;
    const int end = (int)min((int64_t)rg.len, (int64_t)start + p.chunk);
    if (p.splits > 1 && start >= end) return;

    // Q as the second operand: lane l holds head l % 16 and 8 elements of each
    // step.  Elements of step s: 32 s + 8 g .. + 7; for E4M3 keys, whose 16-byte
    // pieces cover two steps, 64 (s / 2) + 16 g + 8 (s % 2) .. + 7.
    auto elem = [&](int s) {
        return E4M3 ? 64 * (s >> 1) + 16 * g4 + 8 * (s & 1) : 32 * s + 8 * g4;
    };
    x8 qf[STEPS];
    {
        const T* row = (const T*)p.q.p + b * p.q.ts + (int64_t)(h0 + min(r16, nh - 1)) * p.q.hs;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int e = elem(s);
            qf[s] = r16 < nh && e < p.D ? *(const x8*)(row + e) : (x8){};
        }
    }

    // Pages and places of a tile's keys.  ALIGNED: the page of each 16 keys, in
    // scalar registers.  Otherwise lane l has that of key l % 32 and the others ask
    // it.  An unusable key (outside [lo, end), or in a hole) gets page -1.
    struct Where {
        int page[ALIGNED ? 2 : 1];
        int at[ALIGNED ? 2 : 1];
    };
    const int32_t* const trow = p.table + b * p.table_stride;
    auto page_of = [&](int key, int& at) {
        const int i = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
        at = key - i * p.page_size;
        return i;
    };
    auto look = [&](int key0) {
        Where w;
        if constexpr (ALIGNED) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = key0 + 16 * h;
                const int i = page_of(key, w.at[h]);
                w.page[h] = key < end ? scalar_int(trow + i) : -1;
            }
        } else {
            const int key = key0 + (lane & 31);
            const int i = page_of(key, w.at[0]);
            w.page[0] = key >= rg.lo && key < end ? trow[i] : -1;
        }
        return w;
    };
    auto settle = [&](Where& w) {
#pragma unroll
        for (int h = 0; h < (ALIGNED ? 2 : 1); ++h)
            if ((uint32_t)w.page[h] >= (uint32_t)p.pages) w.page[h] = -1;
    };

    struct Keys {
        uint32_t k[KI][4];
    };
    struct Values {
        uint32_t v[8][VW];
    };
    // A key's 16-byte piece c lies in LDS at c ^ swz(key): the 16 keys of one operand
    // read then meet 16 different groups of banks.
    constexpr int SH = KL >= 16 ? 0 : KL == 8 ? 1 : 2;
    auto swz = [](int key) { return (key >> SH) & ((KL < 16 ? KL : 16) - 1); };
    char* const ka = lds + wave * KA;
    const int kc = lane % KL, kr = lane / KL;
    // D < DP: pieces of a key past its end are zeros that nothing overwrites; loads
    // past the end of a value row read its beginning for elements nobody stores
    const bool kin = key_piece_in(kc, p.D, ES);
    if (!kin)
#pragma unroll
        for (int i = 0; i < KI; ++i)
            *(i32x4_t*)(ka + (i * KN + kr) * KB + (kc ^ swz(i * KN + kr)) * 16) = (i32x4_t){};
    int vc[VL];
#pragma unroll
    for (int i = 0; i < VL; ++i) vc[i] = value_at(r16, i, p.D, DP, ES);
    // ALIGNED: a lane's offsets from the first of 16 keys (16 token strides are
    // less than 2^31 bytes)
    const uint32_t koff = (uint32_t)kr * (uint32_t)p.k_tok + kc * 16;
    const uint32_t voff = (uint32_t)(4 * g4) * (uint32_t)p.v_tok;
    const char* const kh = p.kc + hk * p.k_head;
    const char* const vh = p.vc + hk * p.v_head;
    // the keys of inner positions 0..7 of this lane in the second product
    auto vkey = [&](int j) { return (j < 4 ? 0 : 16) + 4 * g4 + (j & 3); };
    auto load_keys = [&](Keys& t, const Where& w) {
        if constexpr (ALIGNED) {
            const char* kb[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) kb[h] = kh + max(w.page[h], 0) * p.k_page + w.at[h] * p.k_tok;
            if (kin)
#pragma unroll
                for (int i = 0; i < KI; ++i) {
                    constexpr int HALF = 16 / KN;  // reads of 16 keys
                    load_words<4>(kb[i / HALF] + (i % HALF) * KN * p.k_tok + koff, t.k[i]);
                }
        } else {
            const char* krow[KI];
#pragma unroll
            for (int i = 0; i < KI; ++i)
                krow[i] = kh + max(__shfl(w.page[0], i * KN + kr), 0) * p.k_page +
                          __shfl(w.at[0], i * KN + kr) * p.k_tok + kc * 16;
            if (kin)
#pragma unroll
                for (int i = 0; i < KI; ++i) load_words<4>(krow[i], t.k[i]);
        }
    };
    auto load_values = [&](Values& t, const Where& w) {
        if constexpr (ALIGNED) {
            const char* vb[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) vb[h] = vh + max(w.page[h], 0) * p.v_page + w.at[h] * p.v_tok;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < VL; ++i)
                    load_words<VB / 4>(vb[j >> 2] + (j & 3) * p.v_tok + (voff + vc[i]), t.v[j] + i * (VB / 4));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const char* row = vh + max(__shfl(w.page[0], vkey(j)), 0) * p.v_page +
                                  __shfl(w.at[0], vkey(j)) * p.v_tok;
#pragma unroll
                for (int i = 0; i < VL; ++i) load_words<VB / 4>(row + vc[i], t.v[j] + i * (VB / 4));
            }
        }
    };

    f32x4_t o[VE];
#pragma unroll
    for (int m = 0; m < VE; ++m) o[m] = (f32x4_t){};
    float mx = kNegInf, sum = 0.0f;

    // (`next` asks for the next tile's keys, once the registers of these are free)
    auto compute = [&](Keys& kt, Values& t, const Where& w, int key0, auto&& next) {
        // a tile with unusable keys: their scores become -infinity and, since a
        // probability of 0 times what lies in such a place may be NaN, their
        // values 0
        bool plain;
        if constexpr (ALIGNED) {
            plain = key0 >= rg.lo && key0 + 32 <= end && (w.page[0] | w.page[1]) >= 0;
        } else {
            plain = __ballot(w.page[0] < 0) == 0;
        }
        auto usable = [&](int k32) {
            if constexpr (ALIGNED) {
                const int key = key0 + k32;
                return key >= rg.lo && key < end && (k32 < 16 ? w.page[0] : w.page[1]) >= 0;
            } else {
                return __shfl(w.page[0], k32) >= 0;
            }
        };
        // the keys through LDS, from whole rows into the operand's 16 keys x 16 bytes
        // (the wave's own area: its LDS operations run in order)
        wave_lds_exchange();
        if (kin)
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                const int key = i * KN + kr;
                *(i32x4_t*)(ka + key * KB + (kc ^ swz(key)) * 16) = *(i32x4_t*)kt.k[i];
            }
        wave_lds_exchange();
        next();
        f32x4_t s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = (f32x4_t){};
            const char* row = ka + (16 * h + r16) * KB;
            const int sw = swz(16 * h + r16);
            if constexpr (E4M3) {
#pragma unroll
                for (int st = 0; st < STEPS; st += 2) {
                    const i32x4_t w4 = *(const i32x4_t*)(row + ((2 * st + g4) ^ sw) * 16);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t u[4];
                        u[0] = H::from_fp8(w4[2 * y], false);
                        u[1] = H::from_fp8(w4[2 * y], true);
                        u[2] = H::from_fp8(w4[2 * y + 1], false);
                        u[3] = H::from_fp8(w4[2 * y + 1], true);
                        s[h] = H::mma(__builtin_bit_cast(x8, *(i32x4_t*)u), qf[st + y], s[h]);
                    }
                }
            } else {
#pragma unroll
                for (int st = 0; st < STEPS; ++st)
                    s[h] = H::mma(*(const x8*)(row + ((4 * st + g4) ^ sw) * 16), qf[st], s[h]);
            }
        }
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s[j >> 2][j & 3] * p.scale_log2;
        if (!plain) {
            asm volatile("");  // (a branch: as selects it would run for every tile)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool use = usable(vkey(j));
                x[j] = use ? x[j] : kNegInf;
#pragma unroll
                for (int i = 0; i < VW; ++i) t.v[j][i] = use ? t.v[j][i] : 0u;
            }
        }
        float top = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
        top = max_over_groups(top);
        if (__any(top > mx)) {
            const float m2 = fmaxf(mx, top);
            const float f = m2 == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(mx - m2);
            mx = m2;
            sum *= f;
#pragma unroll
            for (int m = 0; m < VE; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][i] *= f;
        }
        const float m0 = mx == kNegInf ? 0.0f : mx;
        uint32_t pu[4], pl[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float e0 = __builtin_amdgcn_exp2f(x[j] - m0), e1 = __builtin_amdgcn_exp2f(x[j + 1] - m0);
            sum += e0;
            sum += e1;
            H::parts(e0, e1, pu[j / 2], pl[j / 2]);
        }
        const x8 upper = __builtin_bit_cast(x8, *(i32x4_t*)pu), lower = __builtin_bit_cast(x8, *(i32x4_t*)pl);
        // 8 keys x VE elements -> VE operands of 8 keys
#pragma unroll
        for (int m = 0; m < VE; m += 2) {
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                uint32_t v0, v1;
                if constexpr (E4M3) {
                    v0 = H::from_fp8(t.v[2 * jj][m / 4], (m / 2) & 1);
                    v1 = H::from_fp8(t.v[2 * jj + 1][m / 4], (m / 2) & 1);
                } else {
                    v0 = t.v[2 * jj][m / 2];
                    v1 = t.v[2 * jj + 1][m / 2];
                }
                lo[jj] = __builtin_amdgcn_perm(v1, v0, 0x05040100);
                hi[jj] = __builtin_amdgcn_perm(v1, v0, 0x07060302);
            }
            const x8 v0 = __builtin_bit_cast(x8, *(i32x4_t*)lo), v1 = __builtin_bit_cast(x8, *(i32x4_t*)hi);
            o[m] = H::mma(v0, upper, o[m]);
            o[m + 1] = H::mma(v1, upper, o[m + 1]);
            o[m] = H::mma(v0, lower, o[m]);
            o[m + 1] = H::mma(v1, lower, o[m + 1]);
        }
    };

    // The wave's tiles, a round apart.  While one is computed the next one's keys
    // and values are on their way (the values' registers in two sets; those of the
    // keys are free as soon as they are in LDS), and its successor's pages are
    // looked up (asked for before those loads, so that waiting for them is no wait
    // for the loads).
    int key = start + 32 * kw;
    if (key < end) {
        Keys kt;
        Values va, vb;
        Where wa = look(key), wb = look(key + round), wc;
        settle(wa);
        load_keys(kt, wa);
        load_values(va, wa);
        for (;;) {
            settle(wb);
            wc = look(key + 2 * round);
            bool more = key + round < end;
            if (more) load_values(vb, wb);
            compute(kt, va, wa, key, [&] {
                if (more) load_keys(kt, wb);
            });
            if (!more) break;
            key += round;
            settle(wc);
            wa = look(key + 2 * round);
            more = key + round < end;
            if (more) load_values(va, wc);
            compute(kt, vb, wb, key, [&] {
                if (more) load_keys(kt, wc);
            });
            if (!more) break;
            key += round;
            wb = wa;
            wa = wc;
        }
    }

    // ---- the four waves' parts ------------------------------------------------
    __syncthreads();  // (the areas of keys end here)
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    // a NaN among the scores passed by the maximum: as an infinite one it makes
    // every later factor of this part NaN and of the others 0
    if (sum != sum) mx = -kNegInf;
    if (g4 == 0) {
        lm_[wave][r16] = mx;
        ll_[wave][r16] = sum;
    }
    __syncthreads();
    // the largest maximum of the waves that share head hh of the group
    auto head_top = [&](int hh, int q) {
        float t = lm_[hh][q];
        for (int w = hh + p.heads; w < 4; w += p.heads) t = fmaxf(t, lm_[w][q]);
        return t;
    };
    const float f = mx == kNegInf ? 0.0f : 1.0f / H::kLift * __builtin_amdgcn_exp2f(mx - head_top(hw, r16));
    // lane l holds elements (4 g + i) VE + m of head l % 16
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < VE; m += 4) {
            f32x4_t v = {o[m][i] * f, o[m + 1][i] * f, o[m + 2][i] * f, o[m + 3][i] * f};
            if (mx == kNegInf) v = (f32x4_t){};
            *(f32x4_t*)&lo_[wave][r16][(4 * g4 + i) * VE + m] = v;
        }
    __syncthreads();
    for (int x = threadIdx.x; x < p.heads * 16 * (DP / 4); x += 256) {
        const int hh = x / (16 * (DP / 4)), q = x / (DP / 4) % 16, d = x % (DP / 4) * 4;
        if (q >= nh || d >= p.D) continue;
        const float tq = head_top(hh, q);
        f32x4_t a = {};
        float l = 0.0f;
        for (int w = hh; w < 4; w += p.heads) {
            a += *(f32x4_t*)&lo_[w][q][d];
            const float mw = lm_[w][q];
            l += mw == kNegInf ? 0.0f : ll_[w][q] * __builtin_amdgcn_exp2f(mw - tq);
        }
        const int h = (hk - hw + hh) * p.G + qb * 16 + q;
        const int64_t row = (int64_t)b * p.Hq + h;
        if (p.splits > 1) {
            const int64_t at = row * p.splits + split;
            *(f32x4_t*)(p.po + at * p.D + d) = a;
            if (d == 0) {
                p.pml[2 * at] = tq;
                p.pml[2 * at + 1] = l;
            }
        } else {
            const float z = tq == kNegInf ? 0.0f : p.v_scale / l;
            T* out = (T*)p.out.p + b * p.out.ts + (int64_t)h * p.out.hs + d;
            store4<T>(out, a[0] * z, a[1] * z, a[2] * z, a[3] * z);
            if (d == 0 && p.lse)
                p.lse[row] = tq == kNegInf ? kNegInf : 0.6931471805599453f * tq + logf(l);
        }
    }
}

// Joins the chunks of one sequence and query head: DL lanes x 4 elements (blockIdx.z
// picks which), 256 / DL chunks at a time, at most kJoinDeep times.  Bound by
// latency -- the parts come from other XCDs' caches -- so every load of a part is
// under way before the weights that it waits for are computed.
constexpr int kJoinDeep = 8;
template <class T, int DL>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs p) {
    __shared__ float wt[kAttnMaxSplits];
    __shared__ float red[2][4];
    __shared__ __attribute__((aligned(16))) float join[256 / DL][DL * 4];
    constexpr int PARTS = 256 / DL;
    const int h = blockIdx.x, b = blockIdx.y;
    const Range rg = range_of(p, b);
    const int n = (int)(((int64_t)rg.len - rg.base + p.chunk - 1) / p.chunk);
    const int64_t row = (int64_t)b * p.Hq + h;
    const float* ml = p.pml + 2 * row * p.splits;
    const int c = threadIdx.x;
    const int dl = (c % DL) * 4, d = blockIdx.z * DL * 4 + dl, part = c / DL;
    const float m = c < n ? ml[2 * c] : kNegInf;
    const float lc = c < n ? ml[2 * c + 1] : 0.0f;
    f32x4_t v[kJoinDeep];
#pragma unroll
    for (int i = 0; i < kJoinDeep; ++i) {
        const int at = part + i * PARTS;
        v[i] = at < n && d < p.D ? *(const f32x4_t*)(p.po + (row * p.splits + at) * p.D + d) : (f32x4_t){};
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
    for (int i = 0; i < kJoinDeep; ++i) {
        const int at = part + i * PARTS;
        if (at < n) a += wt[at] * v[i];
    }
    *(f32x4_t*)&join[part][dl] = a;
    __syncthreads();
    if (part == 0 && d < p.D) {
#pragma unroll
        for (int i = 1; i < PARTS; ++i) a += *(f32x4_t*)&join[i][dl];
        const float z = top == kNegInf ? 0.0f : p.v_scale / l;
        T* out = (T*)p.out.p + b * p.out.ts + (int64_t)h * p.out.hs + d;
        store4<T>(out, a[0] * z, a[1] * z, a[2] * z, a[3] * z);
        if (d == 0 && p.lse) p.lse[row] = top == kNegInf ? kNegInf : 0.6931471805599453f * top + logf(l);
    }
}

template <class T, int DP, bool E4M3>
hipError_t run(const AttnArgs& a, hipStream_t st) {
    const dim3 grid((uint32_t)a.splits * a.B * (a.Hk / a.heads) * a.qblocks);
    if (a.page_size % 16 == 0)
        hipLaunchKernelGGL((attn_kernel<T, DP, E4M3, true>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((attn_kernel<T, DP, E4M3, false>), grid, dim3(256), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    // a whole row a workgroup where that takes its chunks in kJoinDeep turns,
    // else 32 elements
    if (a.splits <= kJoinDeep * (256 / (DP / 4)))
        hipLaunchKernelGGL((attn_join_kernel<T, DP / 4>), dim3(a.Hq, a.B), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((attn_join_kernel<T, 8>), dim3(a.Hq, a.B, DP / 32), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <class T>
hipError_t by_dim(const AttnArgs& a, bool e4m3, hipStream_t st) {
    switch (head_instance(a.D)) {
    case 64: return e4m3 ? run<T, 64, true>(a, st) : run<T, 64, false>(a, st);
    case 128: return e4m3 ? run<T, 128, true>(a, st) : run<T, 128, false>(a, st);
    default: return e4m3 ? run<T, 256, true>(a, st) : run<T, 256, false>(a, st);
    }
}

}  // namespace

hipError_t launch_paged_attention(const AttnArgs& a, int32_t dtype, bool e4m3, hipStream_t st) {
    return dtype == 1 ? by_dim<__bf16>(a, e4m3, st) : by_dim<_Float16>(a, e4m3, st);
}

}  // namespace tcm
