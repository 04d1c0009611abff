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
// permutations within the lane.  Maximum and sum of a head's softmax live in
// its lanes too: nothing goes through LDS until a workgroup's four waves join.
//
// A workgroup takes a chunk of one sequence's keys for one key-value head, its
// waves 32 keys at a time in turn, the next tile's loads being in flight while
// one is computed.  With more than one chunk the partial results go to the
// workspace and attn_join_kernel joins them.
#include <type_traits>

#include "layer_internal.h"
#include "tcm_device.h"

namespace tcm {

namespace {

constexpr float kNegInf = -__builtin_inff();

template <class T> struct Half16;
template <> struct Half16<__bf16> {
    typedef bf16x8_t x8;
    typedef __bf16 x2 __attribute__((ext_vector_type(2)));
    __device__ static __forceinline__ f32x4_t mma(x8 a, x8 b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    __device__ static __forceinline__ uint32_t from_fp8(uint32_t w, bool hi) {
        return __builtin_bit_cast(uint32_t, hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    }
};
template <> struct Half16<_Float16> {
    typedef f16x8_t x8;
    typedef _Float16 x2 __attribute__((ext_vector_type(2)));
    __device__ static __forceinline__ f32x4_t mma(x8 a, x8 b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    __device__ static __forceinline__ uint32_t from_fp8(uint32_t w, bool hi) {
        return __builtin_bit_cast(uint32_t, hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)
                                               : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    }
};

template <int BYTES> struct Bytes;
template <> struct Bytes<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };
template <> struct Bytes<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <> struct Bytes<4> { typedef uint32_t type __attribute__((ext_vector_type(1))); };

// N words from p (16-byte pieces where N allows)
template <int N>
__device__ __forceinline__ void load_words(const char* p, uint32_t* w) {
    constexpr int B = N % 4 == 0 ? 16 : N * 4;
    typedef typename Bytes<B>::type v_t;
#pragma unroll
    for (int i = 0; i < N * 4 / B; ++i) {
        const v_t v = *(const v_t*)(p + i * B);
#pragma unroll
        for (int j = 0; j < B / 4; ++j) w[i * (B / 4) + j] = v[j];
    }
}

// The keys [lo, end) of sequence b that chunk c covers, and the whole range's
// first tile.
struct Range {
    int base, lo, len;
};
__device__ __forceinline__ Range range_of(const AttnArgs& p, int b) {
    Range r;
    const int64_t room = p.table_stride * (int64_t)p.page_size;
    int len = p.lengths[b];
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
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void attn_kernel(AttnArgs p) {
    typedef Half16<T> H;
    typedef typename H::x8 x8;
    constexpr int ES = E4M3 ? 1 : 2;
    constexpr int STEPS = DP / 32;          // products of 32 over the head
    constexpr int VE = DP / 16;             // elements of a value row a lane holds
    constexpr int KW = E4M3 ? 2 : 4;        // words of a lane's 8 key elements
    constexpr int VW = VE * ES / 4;         // words of a lane's piece of a value row
    __shared__ __attribute__((aligned(16))) float lo_[4][16][DP + 4];
    __shared__ float lm_[4][16], ll_[4][16];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int b = blockIdx.z;
    const int hk = blockIdx.y / p.qblocks, qb = blockIdx.y - hk * p.qblocks;
    const int h0 = hk * p.G + qb * 16, nh = min(16, p.G - qb * 16);
    const Range rg = range_of(p, b);
    const int start = rg.base + (int)blockIdx.x * p.chunk;
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

    // Pages and places of a tile's keys.  ALIGNED: one page and first place per
    // 16 keys.  Otherwise lane l looks up key l % 32 and the others ask it.
    // An unusable key (outside [lo, end), or in a hole) gets page -1.
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
                w.page[h] = key < end ? trow[i] : -1;
                if ((uint32_t)w.page[h] >= (uint32_t)p.pages) w.page[h] = -1;
            }
        } else {
            const int key = key0 + (lane & 31);
            const int i = page_of(key, w.at[0]);
            w.page[0] = key >= rg.lo && key < end ? trow[i] : -1;
            if ((uint32_t)w.page[0] >= (uint32_t)p.pages) w.page[0] = -1;
        }
        return w;
    };

    struct Tile {
        uint32_t k[2][STEPS][KW];
        uint32_t v[8][VW];
    };
    const char* const kh = p.kc + hk * p.k_head;
    const char* const vh = p.vc + hk * p.v_head;
    const bool whole = p.D == DP;
    // the keys of inner positions 0..7 of this lane in the second product
    auto vkey = [&](int j) { return (j < 4 ? 0 : 16) + 4 * g4 + (j & 3); };
    auto load = [&](Tile& t, const Where& w) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int page, at;
            if constexpr (ALIGNED) {
                page = max(w.page[h], 0);
                at = w.at[h] + r16;
            } else {
                page = max(__shfl(w.page[0], r16 + 16 * h), 0);
                at = __shfl(w.at[0], r16 + 16 * h);
            }
            const char* row = kh + page * p.k_page + at * p.k_tok;
            if constexpr (E4M3) {
#pragma unroll
                for (int s = 0; s < STEPS; s += 2) {
                    uint32_t w4[4] = {0, 0, 0, 0};
                    if (whole || elem(s) < p.D) load_words<4>(row + elem(s), w4);
                    t.k[h][s][0] = w4[0], t.k[h][s][1] = w4[1];
                    t.k[h][s + 1][0] = w4[2], t.k[h][s + 1][1] = w4[3];
                }
            } else {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    if (whole || elem(s) < p.D) {
                        load_words<4>(row + 2 * elem(s), t.k[h][s]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) t.k[h][s][i] = 0;
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            int page, at;
            if constexpr (ALIGNED) {
                page = max(w.page[j >> 2], 0);
                at = w.at[j >> 2] + 4 * g4 + (j & 3);
            } else {
                page = max(__shfl(w.page[0], vkey(j)), 0);
                at = __shfl(w.at[0], vkey(j));
            }
            const char* row = vh + page * p.v_page + at * p.v_tok;
            if (whole || r16 * VE < p.D) {
                load_words<VW>(row + r16 * VE * ES, t.v[j]);
            } else {
#pragma unroll
                for (int i = 0; i < VW; ++i) t.v[j][i] = 0;
            }
        }
    };

    f32x4_t o[VE];
#pragma unroll
    for (int m = 0; m < VE; ++m) o[m] = (f32x4_t){};
    float mx = kNegInf, sum = 0.0f;

    auto compute = [&](Tile& t, const Where& w, int key0) {
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
        f32x4_t s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = (f32x4_t){};
#pragma unroll
            for (int st = 0; st < STEPS; ++st) {
                x8 kf;
                if constexpr (E4M3) {
                    uint32_t u[4];
                    u[0] = H::from_fp8(t.k[h][st][0], false);
                    u[1] = H::from_fp8(t.k[h][st][0], true);
                    u[2] = H::from_fp8(t.k[h][st][1], false);
                    u[3] = H::from_fp8(t.k[h][st][1], true);
                    kf = __builtin_bit_cast(x8, *(i32x4_t*)u);
                } else {
                    kf = __builtin_bit_cast(x8, *(i32x4_t*)t.k[h][st]);
                }
                s[h] = H::mma(kf, qf[st], s[h]);
            }
        }
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s[j >> 2][j & 3] * p.scale_log2;
        if (!plain) {
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
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
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
        x8 pf;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float e = __builtin_amdgcn_exp2f(x[j] - m0);
            sum += e;
            pf[j] = (T)e;
        }
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
            o[m] = H::mma(__builtin_bit_cast(x8, *(i32x4_t*)lo), pf, o[m]);
            o[m + 1] = H::mma(__builtin_bit_cast(x8, *(i32x4_t*)hi), pf, o[m + 1]);
        }
    };

    // the wave's tiles, 128 keys apart, two register sets in turn
    int key = start + 32 * wave;
    if (key < end) {
        Tile ta, tb;
        Where wa = look(key), wb;
        load(ta, wa);
        for (;;) {
            const bool more = key + 128 < end;
            if (more) {
                wb = look(key + 128);
                load(tb, wb);
            }
            compute(ta, wa, key);
            if (!more) break;
            key += 128;
            const bool again = key + 128 < end;
            if (again) {
                wa = look(key + 128);
                load(ta, wa);
            }
            compute(tb, wb, key);
            if (!again) break;
            key += 128;
        }
    }

    // ---- the four waves' parts ------------------------------------------------
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
    const float top = fmaxf(fmaxf(lm_[0][r16], lm_[1][r16]), fmaxf(lm_[2][r16], lm_[3][r16]));
    const float f = mx == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mx - top);
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
    for (int x = threadIdx.x; x < 16 * (DP / 4); x += 256) {
        const int q = x / (DP / 4), d = (x - q * (DP / 4)) * 4;
        if (q >= nh || d >= p.D) continue;
        const float tq = fmaxf(fmaxf(lm_[0][q], lm_[1][q]), fmaxf(lm_[2][q], lm_[3][q]));
        f32x4_t a = {};
        float l = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            a += *(f32x4_t*)&lo_[w][q][d];
            const float mw = lm_[w][q];
            l += mw == kNegInf ? 0.0f : ll_[w][q] * __builtin_amdgcn_exp2f(mw - tq);
        }
        const int64_t row = (int64_t)b * p.Hq + h0 + q;
        if (p.splits > 1) {
            const int64_t at = row * p.splits + blockIdx.x;
            *(f32x4_t*)(p.po + at * p.D + d) = a;
            if (d == 0) {
                p.pml[2 * at] = tq;
                p.pml[2 * at + 1] = l;
            }
        } else {
            const float z = tq == kNegInf ? 0.0f : p.v_scale / l;
            T* out = (T*)p.out.p + b * p.out.ts + (int64_t)(h0 + q) * p.out.hs + d;
            store4<T>(out, a[0] * z, a[1] * z, a[2] * z, a[3] * z);
            if (d == 0 && p.lse)
                p.lse[row] = tq == kNegInf ? kNegInf : 0.6931471805599453f * tq + logf(l);
        }
    }
}

// Joins the chunks of one sequence and query head: DL lanes x 4 elements, 256 / DL
// chunks at a time.
template <class T, int DL>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs p) {
    __shared__ float wt[kAttnMaxSplits];
    __shared__ float red[4];
    __shared__ __attribute__((aligned(16))) float join[256 / DL][DL * 4];
    const int h = blockIdx.x, b = blockIdx.y;
    const Range rg = range_of(p, b);
    const int n = (int)(((int64_t)rg.len - rg.base + p.chunk - 1) / p.chunk);
    const int64_t row = (int64_t)b * p.Hq + h;
    const float* ml = p.pml + 2 * row * p.splits;
    const int c = threadIdx.x;
    const float m = c < n ? ml[2 * c] : kNegInf;
    float top = m;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
    if ((c & 63) == 0) red[c >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
    const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - top);
    if (c < kAttnMaxSplits) wt[c] = f;
    float l = c < n ? f * ml[2 * c + 1] : 0.0f;
    if (m == kNegInf) l = 0.0f;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) l += __shfl_xor(l, x);
    if ((c & 63) == 0) red[c >> 6] = l;
    __syncthreads();
    l = red[0] + red[1] + red[2] + red[3];
    const int d = (c % DL) * 4, part = c / DL;
    f32x4_t a = {};
    if (d < p.D)
#pragma unroll 4
        for (int i = part; i < n; i += 256 / DL) {
            const float w = wt[i];
            const f32x4_t v = *(const f32x4_t*)(p.po + (row * p.splits + i) * p.D + d);
            if (w != 0.0f) a += w * v;
        }
    *(f32x4_t*)&join[part][d] = a;
    __syncthreads();
    if (part == 0 && d < p.D) {
#pragma unroll
        for (int i = 1; i < 256 / DL; ++i) a += *(f32x4_t*)&join[i][d];
        const float z = top == kNegInf ? 0.0f : p.v_scale / l;
        T* out = (T*)p.out.p + b * p.out.ts + (int64_t)h * p.out.hs + d;
        store4<T>(out, a[0] * z, a[1] * z, a[2] * z, a[3] * z);
        if (d == 0 && p.lse) p.lse[row] = top == kNegInf ? kNegInf : 0.6931471805599453f * top + logf(l);
    }
}

template <class T, int DP, bool E4M3>
hipError_t run(const AttnArgs& a, hipStream_t st) {
    const dim3 grid(a.splits, a.Hk * a.qblocks, a.B);
    if (a.page_size % 16 == 0)
        hipLaunchKernelGGL((attn_kernel<T, DP, E4M3, true>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((attn_kernel<T, DP, E4M3, false>), grid, dim3(256), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    hipLaunchKernelGGL((attn_join_kernel<T, DP / 4>), dim3(a.Hq, a.B), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <class T>
hipError_t by_dim(const AttnArgs& a, bool e4m3, hipStream_t st) {
    if (a.D <= 64) return e4m3 ? run<T, 64, true>(a, st) : run<T, 64, false>(a, st);
    if (a.D <= 128) return e4m3 ? run<T, 128, true>(a, st) : run<T, 128, false>(a, st);
    return e4m3 ? run<T, 256, true>(a, st) : run<T, 256, false>(a, st);
}

}  // namespace

hipError_t launch_paged_attention(const AttnArgs& a, int32_t dtype, bool e4m3, hipStream_t st) {
    return dtype == 1 ? by_dim<__bf16>(a, e4m3, st) : by_dim<_Float16>(a, e4m3, st);
}

}  // namespace tcm
