// Norm and rotation of query and key heads: forward (dense, or into a paged
// cache) and backward.
//
// A head x of D elements becomes n = x w r, r = (mean(x^2) + eps)^-1/2, whose
// pairs are turned by position * inv_freq.  All of it is bound by memory: a head
// is read once and written once.  L lanes hold one head, 2 E elements each: E
// at `a` and E at `b`, chosen so that a lane holds whole pairs (half layout:
// a = E u, b = rot / 2 + E u; interleaved: 2 E consecutive elements), so the
// rotation needs no other lane and the norm one sum over L lanes.  With E = 8
// every access is 16 bytes and a head's two halves are contiguous over its
// lanes; and as what is done once a head and lane -- the sum, the root, the
// addresses -- is half of the instructions, few lanes a head count as much
// (8191 tokens of 32 + 8 + 8 heads of 128, E4M3 cache: 42 us, 4.3 TB/s, and 77 with
// E = 4; backwards 8192 tokens of 32 + 8 heads 52 us, 4.9 TB/s, and 5 for the sums).
// The angles of a workgroup's tokens are computed once, by its threads, into
// LDS: position * inv_freq in two times 64 bits, reduced to one turn there and only then
// rounded, so a position near 2^31 is as good as one near 0 and no table has to
// be read.
#include <type_traits>

#include "layer_internal.h"
#include "tcm_device.h"

namespace tcm {

namespace {

// E elements at p in one access
template <int E, class T>
__device__ __forceinline__ void load_e(const T* p, float* x) {
    typedef T vec __attribute__((ext_vector_type(E)));
    const vec v = *(const vec*)p;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = (float)v[i];
}
template <int E, class T>
__device__ __forceinline__ void store_e(T* p, const float* x) {
    typedef T vec __attribute__((ext_vector_type(E)));
    vec v;
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = convert_out<T>(x[i]);
    *(vec*)p = v;
}
// E elements of a weight (fp32 or T); ones where there is none
template <int E, class T>
__device__ __forceinline__ void load_w(const void* w, int f32, int at, float* x) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = 1.0f;
    } else if (!f32) {
        load_e<E>((const T*)w + at, x);
    } else {
        constexpr int V = E < 4 ? E : 4;
#pragma unroll
        for (int i = 0; i < E; i += V) load_e<V>((const float*)w + at + i, x + i);
    }
}

// y / scale clamped to +-448, NaN kept.  With 2^-e y, clamped, and the scale's mantissa m
// nothing in the quotient leaves fp32's range, so the residue y - q m is exact and
// corrects q = y (1 / m) to the quotient rounded to nearest: a product with a rounded
// reciprocal alone falls on the wrong side of a tie of E4M3 now and then.  (8191 tokens
// into an E4M3 cache take 42.7 us, and 44.6 with the compiler's division.)
__device__ __forceinline__ float e4m3_quotient(float y, const E4m3Scale& s) {
    const float x = __builtin_ldexpf(y, -s.e);
    const float c = x != x ? x : __builtin_amdgcn_fmed3f(x, -s.top, s.top);
    const float q = c * s.inv;
    return fmaf(fmaf(-q, s.m, c), s.inv, q);
}
// E4M3 of values within its range (or NaN)
template <int E>
__device__ __forceinline__ void store_e4m3(unsigned char* p, const float* x) {
    if constexpr (E == 1) {
        p[0] = (unsigned char)__builtin_amdgcn_cvt_pk_fp8_f32(x[0], 0.0f, 0, false);
    } else {
        typedef int vec __attribute__((ext_vector_type(E / 4)));
        vec v;
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const float* y = x + 4 * i;
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
            v[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
        }
        *(vec*)p = v;
    }
}

// Sum over the L lanes of a head (every lane gets it): within 16 lanes by
// register-lane permutations, beyond them by shuffles.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ float head_sum(float x) {
    x += dpp<0xB1>(x);              // lanes 1, 0, 3, 2 of a quad
    x += dpp<0x4E>(x);              // 2, 3, 0, 1
    if constexpr (L >= 8) x += dpp<0x141>(x);   // mirrored within 8
    if constexpr (L >= 16) x += dpp<0x140>(x);  // mirrored within 16
    if constexpr (L >= 32) x += __shfl_xor(x, 16);
    if constexpr (L >= 64) x += __shfl_xor(x, 32);
    return x;
}

// 1 / sqrt(x): the hardware's approximation (1 ulp) and one Newton step
__device__ __forceinline__ float inv_sqrt(float x) {
    const float r = __builtin_amdgcn_rsqf(x);
    const float e = 0.5f - 0.5f * x * r * r;
    // (zero, infinite and NaN x have no step)
    return e == e ? r + r * e : r;
}

// The unit u of a head: where its elements are, and the first of its pairs.
struct Unit {
    int a, b, f;
    bool live, turn;
};
template <int E, bool INTER>
__device__ __forceinline__ Unit unit_of(int u, int D, int rot) {
    Unit x;
    x.live = 2 * E * u < D;
    x.turn = 2 * E * u < rot;
    const bool half = x.turn && !INTER;
    x.a = half ? E * u : 2 * E * u;
    x.b = half ? rot / 2 + E * u : 2 * E * u + E;
    x.f = E * u;
    return x;
}

// cos and sin of the angles of tokens t0 .. t0 + nt - 1 into cs[0], cs[1]
__device__ __forceinline__ void angles(const RopeArgs& p, int t0, int nt, float (*cs)[kRopeTrig]) {
    const int half = p.rot >> 1;
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int t = i / half, j = i - t * half;
        // The part of a turn, with what each product's rounding leaves: as one double 3e8
        // turns are off by up to 4e-7 radians, these sums by less than 1e-14.  1 / (2 pi)
        // is the sum of two doubles.
        constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnRest = -0x1.6b01ec5417056p-57;
        const double pos = (double)p.pos[t0 + t], f = p.inv_freq[j];
        const double angle = pos * f, angle_rest = fma(pos, f, -angle);
        const double turns = fma(angle, kTurn, -rint(angle * kTurn)) + (angle * kTurnRest + angle_rest * kTurn);
        float s, c;
        sincospif((float)(2.0 * turns), &s, &c);
        cs[0][i] = c * p.factor;
        cs[1][i] = s * p.factor;
    }
}

// E floats of LDS at a multiple of E, in 16-byte reads where E allows
template <int E>
__device__ __forceinline__ void lds_floats(const float* p, float* x) {
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const f32x4_t v = *(const f32x4_t*)(p + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = p[i];
    }
}

// (a, b) turned by the angles c + i s; sign -1 turns back
template <int E, bool INTER>
__device__ __forceinline__ void turn(float* a, float* b, const float* c, const float* s, float sign) {
    if constexpr (INTER && E > 1) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], sn = sign * s[i];
            a[2 * i] = x * c[i] - y * sn;
            a[2 * i + 1] = y * c[i] + x * sn;
            const float z = b[2 * i], w = b[2 * i + 1], sm = sign * s[E / 2 + i];
            b[2 * i] = z * c[E / 2 + i] - w * sm;
            b[2 * i + 1] = w * c[E / 2 + i] + z * sm;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float x = a[i], y = b[i], sn = sign * s[i];
            a[i] = x * c[i] - y * sn;
            b[i] = y * c[i] + x * sn;
        }
    }
}

// (token, head) of an item, and of the one `by` further: one division at the start
struct Item {
    int t, h, dt, dh, H;
    __device__ __forceinline__ Item(int item, int by, int H_)
        : t(item / H_), h(item - item / H_ * H_), dt(by / H_), dh(by - by / H_ * H_), H(H_) {}
    __device__ __forceinline__ void step() {
        t += dt;
        h += dh;
        if (h >= H) h -= H, ++t;
    }
};

// ---- forward ------------------------------------------------------------------
// A workgroup takes p.tb tokens and, of their items -- query heads of all tokens, then
// key heads, then value heads -- p.per; 256 / L at a time, the next ones being loaded
// while these are computed.
template <class T, int L, int E, int NU, bool INTER>
__global__ __launch_bounds__(256) void norm_rope_kernel(RopeArgs p) {
    __shared__ __attribute__((aligned(16))) float cs[2][kRopeTrig];
    // the tokens' places in the cache (read beside the heads, a slot would be
    // waited for with all the reads that went out before it)
    __shared__ int32_t slot_of[kRopeTokens];
    constexpr int GROUPS = 256 / L;
    const int group = threadIdx.x / L, ul = threadIdx.x % L;
    const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.T - t0);
    const int H = p.Hq + p.Hk + p.Hv;
    const int first = blockIdx.y * p.per, last = min(nt * H, first + p.per);
    if (first >= last) return;
    if (p.slots && threadIdx.x < nt) slot_of[threadIdx.x] = p.slots[t0 + threadIdx.x];
    angles(p, t0, nt, cs);
    __syncthreads();
    Unit un[NU];
#pragma unroll
    for (int n = 0; n < NU; ++n) un[n] = unit_of<E, INTER>(ul + n * L, p.D, p.rot);

    // 0 query, 1 key, 2 value heads; items from `base` on
    auto heads = [&](auto WHICH, int base) {
        constexpr int which = decltype(WHICH)::value;
        const int Hw = which == 0 ? p.Hq : which == 1 ? p.Hk : p.Hv;
        const HeadView& v = which == 0 ? p.q : which == 1 ? p.k : p.v;
        const int from = max(first, base) - base, to = min(last, base + nt * Hw) - base;
        if (from + group >= to) return;
        float w[NU][2 * E];
        if (which < 2 && p.norm)
#pragma unroll
            for (int n = 0; n < NU; ++n)
                if (un[n].live) {
                    load_w<E, T>(which ? p.wk : p.wq, p.w_f32, un[n].a, w[n]);
                    load_w<E, T>(which ? p.wk : p.wq, p.w_f32, un[n].b, w[n] + E);
                }
        float x[NU][2 * E];
        auto load = [&](const Item& it) {
            const T* row = (const T*)v.p + (int64_t)(t0 + it.t) * v.ts + it.h * v.hs;
#pragma unroll
            for (int n = 0; n < NU; ++n) {
                if (un[n].live) {
                    load_e<E>(row + un[n].a, x[n]);
                    load_e<E>(row + un[n].b, x[n] + E);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * E; ++i) x[n][i] = 0.0f;
                }
            }
        };
        Item it(from + group, GROUPS, Hw);
        load(it);
        for (int i0 = from + group; i0 < to; i0 += GROUPS) {
            float y[NU][2 * E];
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int i = 0; i < 2 * E; ++i) y[n][i] = x[n][i];
            const int now_t = it.t, now_h = it.h;
            it.step();
            if (i0 + GROUPS < to) load(it);
            if (which < 2) {
                if (p.norm) {
                    float ss = 0.0f;
#pragma unroll
                    for (int n = 0; n < NU; ++n)
#pragma unroll
                        for (int i = 0; i < 2 * E; ++i) ss += y[n][i] * y[n][i];
                    const float r = inv_sqrt(head_sum<L>(ss) * p.inv_d + p.eps);
#pragma unroll
                    for (int n = 0; n < NU; ++n)
#pragma unroll
                        for (int i = 0; i < 2 * E; ++i) y[n][i] *= r * w[n][i];
                }
#pragma unroll
                for (int n = 0; n < NU; ++n)
                    if (un[n].turn) {
                        float c[E], sn[E];
                        const int at = now_t * (p.rot >> 1) + un[n].f;
                        lds_floats<E>(&cs[0][at], c);
                        lds_floats<E>(&cs[1][at], sn);
                        turn<E, INTER>(y[n], y[n] + E, c, sn, 1.0f);
                    }
            }
            if (which == 0 || !p.slots) {
                const HeadView& o = which ? p.ko : p.qo;
                T* row = (T*)o.p + (int64_t)(t0 + now_t) * o.ts + now_h * o.hs;
#pragma unroll
                for (int n = 0; n < NU; ++n)
                    if (un[n].live) {
                        store_e<E>(row + un[n].a, y[n]);
                        store_e<E>(row + un[n].b, y[n] + E);
                    }
                continue;
            }
            const int64_t slot = slot_of[now_t];
            if (slot < 0 || slot >= p.num_slots) continue;
            const int page = p.page_shift >= 0 ? (int)slot >> p.page_shift : (int)slot / p.page_size;
            const int at = (int)slot - page * p.page_size;
            char* row = which == 1 ? (char*)p.kc + page * p.k_page + at * p.k_tok + now_h * p.k_head
                                   : (char*)p.vc + page * p.v_page + at * p.v_tok + now_h * p.v_head;
            const E4m3Scale& scale = which == 1 ? p.k_scale : p.v_scale;
#pragma unroll
            for (int n = 0; n < NU; ++n)
                if (un[n].live) {
                    if (p.cache_e4m3) {
                        float z[2 * E];
#pragma unroll
                        for (int i = 0; i < 2 * E; ++i) z[i] = e4m3_quotient(y[n][i], scale);
                        store_e4m3<E>((unsigned char*)row + un[n].a, z);
                        store_e4m3<E>((unsigned char*)row + un[n].b, z + E);
                    } else {
                        store_e<E>((T*)row + un[n].a, y[n]);
                        store_e<E>((T*)row + un[n].b, y[n] + E);
                    }
                }
        }
    };
    heads(std::integral_constant<int, 0>{}, 0);
    heads(std::integral_constant<int, 1>{}, nt * p.Hq);
    if (p.Hv > 0) heads(std::integral_constant<int, 2>{}, nt * (p.Hq + p.Hk));
}

// ---- backward -----------------------------------------------------------------
// With h = x r and g = w rot^T(dy): dx = r (g - h mean(g h)), dw = sum of
// rot^T(dy) h.  Both sums of a head, x^2 and g x, are taken in one pass over its
// registers (mean(g h) = r mean(g x)).  A workgroup walks token blocks gridDim.x
// apart and keeps its part of the weight gradients in registers, query heads
// first and then key heads of a block, so a lane adds to one of the two; the
// parts are joined over the workgroup in LDS at the end, over workgroups by
// norm_rope_dw_kernel, in a fixed order both.
template <class T, int L, int E, int NU, bool INTER>
__global__ __launch_bounds__(256) void norm_rope_bwd_kernel(RopeArgs p) {
    __shared__ __attribute__((aligned(16))) float cs[2][2][kRopeTrig];
    constexpr int GROUPS = 256 / L;
    __shared__ float join[256 * 2 * E * NU];
    const int group = threadIdx.x / L, ul = threadIdx.x % L;
    const int blocks = (p.T + p.tb - 1) / p.tb;
    Unit un[NU];
#pragma unroll
    for (int n = 0; n < NU; ++n) un[n] = unit_of<E, INTER>(ul + n * L, p.D, p.rot);
    float w[2][NU][2 * E], dw[2][NU][2 * E];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
#pragma unroll
        for (int i = 0; i < 2 * E; ++i) dw[0][n][i] = dw[1][n][i] = 0.0f, w[0][n][i] = w[1][n][i] = 1.0f;
        if (p.norm && un[n].live) {
            load_w<E, T>(p.wq, p.w_f32, un[n].a, w[0][n]);
            load_w<E, T>(p.wq, p.w_f32, un[n].b, w[0][n] + E);
            load_w<E, T>(p.wk, p.w_f32, un[n].a, w[1][n]);
            load_w<E, T>(p.wk, p.w_f32, un[n].b, w[1][n] + E);
        }
    }
    auto heads = [&](int t0, int nt, const float (*c2)[kRopeTrig], auto WHICH) {
        constexpr int which = decltype(WHICH)::value;
        const int H = which ? p.Hk : p.Hq;
        const HeadView& xv = which ? p.k : p.q;
        const HeadView& dyv = which ? p.dko : p.dqo;
        const HeadView& dxv = which ? p.ko : p.qo;
        if (group >= nt * H) return;
        Item it(group, GROUPS, H);
        for (int item = group; item < nt * H; item += GROUPS, it.step()) {
            const int t = it.t, h = it.h;
            const T* xr = (const T*)xv.p + (int64_t)(t0 + t) * xv.ts + h * xv.hs;
            const T* dyr = (const T*)dyv.p + (int64_t)(t0 + t) * dyv.ts + h * dyv.hs;
            float x[NU][2 * E], dy[NU][2 * E];
            float ss = 0.0f, gx = 0.0f;
#pragma unroll
            for (int n = 0; n < NU; ++n) {
                if (un[n].live) {
                    load_e<E>(dyr + un[n].a, dy[n]);
                    load_e<E>(dyr + un[n].b, dy[n] + E);
                    if (p.norm) {
                        load_e<E>(xr + un[n].a, x[n]);
                        load_e<E>(xr + un[n].b, x[n] + E);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * E; ++i) x[n][i] = dy[n][i] = 0.0f;
                }
                if (un[n].turn) {
                    float c[E], s[E];
                    const int at = t * (p.rot >> 1) + un[n].f;
                    lds_floats<E>(&c2[0][at], c);
                    lds_floats<E>(&c2[1][at], s);
                    turn<E, INTER>(dy[n], dy[n] + E, c, s, -1.0f);
                }
            }
            if (p.norm) {
#pragma unroll
                for (int n = 0; n < NU; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * E; ++i) {
                        ss += x[n][i] * x[n][i];
                        gx += dy[n][i] * w[which][n][i] * x[n][i];
                    }
                ss = head_sum<L>(ss);
                gx = head_sum<L>(gx);
                const float r = inv_sqrt(ss * p.inv_d + p.eps);
                const float m = r * r * gx * p.inv_d;  // mean(g h) r
#pragma unroll
                for (int n = 0; n < NU; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * E; ++i) {
                        dw[which][n][i] += dy[n][i] * (x[n][i] * r);
                        dy[n][i] = r * (dy[n][i] * w[which][n][i] - x[n][i] * m);
                    }
            }
            T* dxr = (T*)dxv.p + (int64_t)(t0 + t) * dxv.ts + h * dxv.hs;
#pragma unroll
            for (int n = 0; n < NU; ++n)
                if (un[n].live) {
                    store_e<E>(dxr + un[n].a, dy[n]);
                    store_e<E>(dxr + un[n].b, dy[n] + E);
                }
        }
    };
    int buf = 0;
    for (int b = blockIdx.x; b < blocks; b += gridDim.x, buf ^= 1) {
        const int t0 = b * p.tb, nt = min(p.tb, p.T - t0);
        // (the other buffer may still be read: one barrier a block is enough)
        angles(p, t0, nt, cs[buf]);
        __syncthreads();
        heads(t0, nt, cs[buf], std::integral_constant<int, 0>{});
        heads(t0, nt, cs[buf], std::integral_constant<int, 1>{});
    }
    if (!p.partial) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NU; ++n)
            if (un[n].live)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    join[group * p.D + un[n].a + i] = dw[which][n][i];
                    join[group * p.D + un[n].b + i] = dw[which][n][E + i];
                }
        __syncthreads();
        for (int d = threadIdx.x; d < p.D; d += 256) {
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) s += join[g * p.D + d];
            p.partial[((int64_t)blockIdx.x * 2 + which) * p.D + d] = s;
        }
    }
}

// The sums of `rows` partial weight gradients: 16 columns a workgroup, 16
// threads a column.
__global__ __launch_bounds__(256) void norm_rope_dw_kernel(const float* partial, int rows, int D,
                                                           float* dwq, float* dwk) {
    __shared__ float join[16][17];
    const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
    const int col = blockIdx.x * 16 + c;
    float s = 0.0f;
#pragma unroll 8
    for (int r = part; r < rows; r += 16) s += partial[(int64_t)r * 2 * D + col];
    join[part][c] = s;
    __syncthreads();
    if (threadIdx.x < 16) {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a += join[i][c];
        float* dw = col < D ? dwq : dwk;
        if (dw) dw[col < D ? col : col - D] = a;
    }
}

int cdiv_i(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// f(lanes, elements, units, layout) of the instance for these sizes: E = 8 where
// pairs and what is not rotated come in groups of eight (rot_dim and head_dim
// multiples of 16), E = 4 where pairs come in fours, else pair by pair.
// (WIDE: E = 8 is for the forward pass; the backward one keeps twice the heads and
// the weights' sums in registers, and takes 69 us with it and 58 without for 8192
// tokens of 32 + 8 heads of 128.)
template <bool WIDE, class F>
hipError_t by_shape(int D, int rot, bool inter, F&& f) {
    auto with = [&](auto L, auto E, auto NU) {
        return inter ? f(L, E, NU, std::true_type{}) : f(L, E, NU, std::false_type{});
    };
    std::integral_constant<int, 1> i1;
    std::integral_constant<int, 2> i2;
    std::integral_constant<int, 4> i4;
    std::integral_constant<int, 8> i8;
    if constexpr (WIDE) {
        if (rot % 16 == 0 && D % 16 == 0) {
            if (D <= 64) return with(i4, i8, i1);
            if (D <= 128) return with(i8, i8, i1);
            return with(std::integral_constant<int, 16>{}, i8, i1);
        }
    }
    if (rot % 8 != 0) return with(std::integral_constant<int, 64>{}, i1, i2);
    if (D <= 64) return with(i8, i4, i1);
    if (D <= 128) return with(std::integral_constant<int, 16>{}, i4, i1);
    return with(std::integral_constant<int, 32>{}, i4, i1);
}

template <class T>
hipError_t forward(RopeArgs a, bool inter, hipStream_t st) {
    return by_shape<true>(a.D, a.rot, inter, [&](auto L, auto E, auto NU, auto INTER) {
        constexpr int groups = 256 / decltype(L)::value;
        const int H = a.Hq + a.Hk + a.Hv;
        // Tokens a workgroup: as many as leave four workgroups for every compute
        // unit, since each begins with the angles and its first reads (8191 tokens
        // of 32 + 8 + 8 heads of 128: with eight 6 us more, with 16 13 more, with two 3);
        // with small heads until its items fill its lanes, while every compute unit
        // has a workgroup.
        a.tb = 1;
        while (2 * a.tb * (a.rot / 2) <= kRopeTrig && 2 * a.tb <= kRopeTokens &&
               cdiv_i(a.T, 2 * a.tb) >= (a.tb * H < groups ? 256 : 1024))
            a.tb *= 2;
        // few workgroups: a token block's heads are spread over several
        const int steps = cdiv_i((int64_t)a.tb * H, groups), blocks = cdiv_i(a.T, a.tb);
        int y = cdiv_i(1024, blocks);
        if (y > steps) y = steps;
        a.per = cdiv_i(steps, y) * groups;
        const dim3 grid(blocks, cdiv_i((int64_t)a.tb * H, a.per));
        hipLaunchKernelGGL((norm_rope_kernel<T, decltype(L)::value, decltype(E)::value,
                                             decltype(NU)::value, decltype(INTER)::value>),
                           grid, dim3(256), 0, st, a);
        return hipGetLastError();
    });
}

template <class T>
hipError_t backward(RopeArgs a, bool inter, hipStream_t st) {
    return by_shape<false>(a.D, a.rot, inter, [&](auto L, auto E, auto NU, auto INTER) {
        constexpr int groups = 256 / decltype(L)::value;
        // tokens a step: until the key heads of a block fill the lanes too,
        // while there are steps enough for every workgroup's first
        a.tb = 1;
        while ((int64_t)a.tb * (a.Hk > 0 ? a.Hk : a.Hq) < groups && 2 * a.tb * (a.rot / 2) <= kRopeTrig &&
               cdiv_i(a.T, 2 * a.tb) >= 512)
            a.tb *= 2;
        const int blocks = cdiv_i(a.T, a.tb);
        const int grid = blocks < kRopeBwdGrid ? blocks : kRopeBwdGrid;
        if (grid > 0)
            hipLaunchKernelGGL((norm_rope_bwd_kernel<T, decltype(L)::value, decltype(E)::value,
                                                     decltype(NU)::value, decltype(INTER)::value>),
                               dim3(grid), dim3(256), 0, st, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || !a.partial) return e;
        hipLaunchKernelGGL(norm_rope_dw_kernel, dim3(2 * a.D / 16), dim3(256), 0, st, a.partial, grid,
                           a.D, a.dwq, a.dwk);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_norm_rope(const RopeArgs& a, int32_t dtype, int32_t layout, hipStream_t st) {
    return dtype == 1 ? forward<__bf16>(a, layout == 1, st) : forward<_Float16>(a, layout == 1, st);
}

hipError_t launch_norm_rope_bwd(const RopeArgs& a, int32_t dtype, int32_t layout, hipStream_t st) {
    return dtype == 1 ? backward<__bf16>(a, layout == 1, st) : backward<_Float16>(a, layout == 1, st);
}

}  // namespace tcm
