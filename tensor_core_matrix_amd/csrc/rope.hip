// Norm and rotation of query and key heads: forward (dense, or into a paged
// cache) and backward.
//
// A head x of D elements becomes n = x w r, r = (mean(x^2) + eps)^-1/2, whose
// pairs are turned by position * inv_freq.  All of it is bound by memory: a head
// is read once and written once.  L lanes hold one head, 2 E elements each: E
// at `a` and E at `b`, chosen so that a lane holds whole pairs (half layout:
// a = E u, b = rot / 2 + E u; interleaved: 2 E consecutive elements), so the
// rotation needs no other lane and the norm one sum over L lanes.  With E = 4
// every access is 8 bytes and a head's two halves are contiguous over its
// lanes.  The angles of a workgroup's tokens are computed once, by the threads
// of the workgroup, into LDS: position * inv_freq in 64 bits, reduced to one
// turn there and only then rounded, so a position near 2^31 is as good as one
// near 0 and no table has to be read.
#include <stdlib.h>
#include <type_traits>

#include "layer_internal.h"
#include "tcm_device.h"

namespace tcm {

namespace {

template <class T>
__device__ __forceinline__ float to_f(T x) { return (float)x; }

// E elements at p (E == 4: one 8-byte access)
template <int E, class T>
__device__ __forceinline__ void load_e(const T* p, float* x) {
    if constexpr (E == 4) {
        typedef T t4 __attribute__((ext_vector_type(4)));
        const t4 v = *(const t4*)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)v[i];
    } else {
        x[0] = (float)p[0];
    }
}
template <int E, class T>
__device__ __forceinline__ void store_e(T* p, const float* x) {
    if constexpr (E == 4) {
        store4<T>(p, x[0], x[1], x[2], x[3]);
    } else {
        p[0] = convert_out<T>(x[0]);
    }
}
// E elements of a weight (fp32 or T); ones where there is none
template <int E, class T>
__device__ __forceinline__ void load_w(const void* w, int f32, int at, float* x) {
#pragma unroll
    for (int i = 0; i < E; ++i)
        x[i] = !w ? 1.0f : f32 ? ((const float*)w)[at + i] : (float)((const T*)w)[at + i];
}

// E4M3 of x, saturated at +-448, NaN kept
__device__ __forceinline__ float e4m3_range(float x) {
    return x != x ? x : __builtin_amdgcn_fmed3f(x, -448.0f, 448.0f);
}
template <int E>
__device__ __forceinline__ void store_e4m3(unsigned char* p, const float* x) {
    if constexpr (E == 4) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(x[0]), e4m3_range(x[1]), 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(x[2]), e4m3_range(x[3]), v, true);
        *(int*)p = v;
    } else {
        p[0] = (unsigned char)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(x[0]), 0.0f, 0, false);
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
    x += dpp<0x141>(x);             // mirrored within 8
    if constexpr (L >= 16) x += dpp<0x140>(x);  // mirrored within 16
    if constexpr (L >= 32) x += __shfl_xor(x, 16);
    if constexpr (L >= 64) x += __shfl_xor(x, 32);
    return x;
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
        double turns = (double)p.pos[t0 + t] * p.inv_freq[j] * 0.15915494309189535;  // 1 / (2 pi)
        turns -= rint(turns);
        float s, c;
        sincospif((float)(2.0 * turns), &s, &c);
        cs[0][i] = c * p.factor;
        cs[1][i] = s * p.factor;
    }
}

// (a, b) turned by the angles c + i s; sign -1 turns back
template <int E, bool INTER>
__device__ __forceinline__ void turn(float* a, float* b, const float* c, const float* s, float sign) {
    if constexpr (INTER && E == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], sn = sign * s[i];
            a[2 * i] = x * c[i] - y * sn;
            a[2 * i + 1] = y * c[i] + x * sn;
            const float z = b[2 * i], w = b[2 * i + 1], sm = sign * s[2 + i];
            b[2 * i] = z * c[2 + i] - w * sm;
            b[2 * i + 1] = w * c[2 + i] + z * sm;
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

// ---- forward ------------------------------------------------------------------
// A workgroup takes p.tb tokens and, of their (token, head) items, p.per; 256 / L
// at a time, the next ones being loaded while these are computed.
template <class T, int L, int E, int NU, bool INTER>
__global__ __launch_bounds__(256) void norm_rope_kernel(RopeArgs p) {
    __shared__ float cs[2][kRopeTrig];
    constexpr int GROUPS = 256 / L;
    const int group = threadIdx.x / L, ul = threadIdx.x % L;
    const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.T - t0);
    const int H = p.Hq + p.Hk + p.Hv;
    const int first = blockIdx.y * p.per, last = min(nt * H, first + p.per);
    if (first >= last) return;
    Unit un[NU];
#pragma unroll
    for (int n = 0; n < NU; ++n) un[n] = unit_of<E, INTER>(ul + n * L, p.D, p.rot);

    // the heads of two items, one GROUPS after the other
    constexpr int IN = 2;
    float x[IN][NU][2 * E];
    auto load = [&](int item0) {
#pragma unroll
        for (int z = 0; z < IN; ++z) {
            const int item = item0 + z * GROUPS;
            if (item >= last) continue;
            const int t = item / H, h = item - t * H;
            const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hk;
            const HeadView& v = is_q ? p.q : is_k ? p.k : p.v;
            const int hh = is_q ? h : is_k ? h - p.Hq : h - p.Hq - p.Hk;
            const T* row = (const T*)v.p + (int64_t)(t0 + t) * v.ts + hh * v.hs;
#pragma unroll
            for (int n = 0; n < NU; ++n) {
                if (un[n].live) {
                    load_e<E>(row + un[n].a, x[z][n]);
                    load_e<E>(row + un[n].b, x[z][n] + E);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * E; ++i) x[z][n][i] = 0.0f;
                }
            }
        }
    };
    int item0 = first + group;
    load(item0);
    float wq[NU][2 * E], wk[NU][2 * E];
    if (p.norm) {
#pragma unroll
        for (int n = 0; n < NU; ++n)
            if (un[n].live) {
                load_w<E, T>(p.wq, p.w_f32, un[n].a, wq[n]);
                load_w<E, T>(p.wq, p.w_f32, un[n].b, wq[n] + E);
                load_w<E, T>(p.wk, p.w_f32, un[n].a, wk[n]);
                load_w<E, T>(p.wk, p.w_f32, un[n].b, wk[n] + E);
            }
    }
    angles(p, t0, nt, cs);
    __syncthreads();

    auto finish = [&](int item, float (&y)[NU][2 * E]) {
        const int t = item / H, h = item - t * H;
        const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hk;
        if (is_q || is_k) {
            if (p.norm) {
                float ss = 0.0f;
#pragma unroll
                for (int n = 0; n < NU; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * E; ++i) ss += y[n][i] * y[n][i];
                ss = head_sum<L>(ss);
                const float r = 1.0f / sqrtf(ss / (float)p.D + p.eps);
#pragma unroll
                for (int n = 0; n < NU; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * E; ++i) y[n][i] *= r * (is_q ? wq[n][i] : wk[n][i]);
            }
#pragma unroll
            for (int n = 0; n < NU; ++n)
                if (un[n].turn) {
                    float c[E], s[E];
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        c[i] = cs[0][t * (p.rot >> 1) + un[n].f + i];
                        s[i] = cs[1][t * (p.rot >> 1) + un[n].f + i];
                    }
                    turn<E, INTER>(y[n], y[n] + E, c, s, 1.0f);
                }
        }
        if (is_q || !p.slots) {
            const HeadView& o = is_q ? p.qo : p.ko;
            T* row = (T*)o.p + (int64_t)(t0 + t) * o.ts + (is_q ? h : h - p.Hq) * o.hs;
#pragma unroll
            for (int n = 0; n < NU; ++n)
                if (un[n].live) {
                    store_e<E>(row + un[n].a, y[n]);
                    store_e<E>(row + un[n].b, y[n] + E);
                }
            return;
        }
        const int64_t slot = p.slots[t0 + t];
        if (slot < 0 || slot >= p.num_slots) return;
        const int page = (int)slot / p.page_size, at = (int)slot - page * p.page_size;
        char* row = is_k ? (char*)p.kc + page * p.k_page + at * p.k_tok + (h - p.Hq) * p.k_head
                         : (char*)p.vc + page * p.v_page + at * p.v_tok +
                               (h - p.Hq - p.Hk) * p.v_head;
        const float inv = is_k ? p.k_inv : p.v_inv;
#pragma unroll
        for (int n = 0; n < NU; ++n)
            if (un[n].live) {
                if (p.cache_e4m3) {
                    float z[2 * E];
#pragma unroll
                    for (int i = 0; i < 2 * E; ++i) z[i] = y[n][i] * inv;
                    store_e4m3<E>((unsigned char*)row + un[n].a, z);
                    store_e4m3<E>((unsigned char*)row + un[n].b, z + E);
                } else {
                    store_e<E>((T*)row + un[n].a, y[n]);
                    store_e<E>((T*)row + un[n].b, y[n] + E);
                }
            }
    };
    for (; item0 < last; item0 += IN * GROUPS) {
        float y[IN][NU][2 * E];
#pragma unroll
        for (int z = 0; z < IN; ++z)
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int i = 0; i < 2 * E; ++i) y[z][n][i] = x[z][n][i];
        load(item0 + IN * GROUPS);
#pragma unroll
        for (int z = 0; z < IN; ++z)
            if (item0 + z * GROUPS < last) finish(item0 + z * GROUPS, y[z]);
    }
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
    __shared__ float cs[2][2][kRopeTrig];
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
        for (int item = group; item < nt * H; item += GROUPS) {
            const int t = item / H, h = item - t * H;
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
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        c[i] = c2[0][t * (p.rot >> 1) + un[n].f + i];
                        s[i] = c2[1][t * (p.rot >> 1) + un[n].f + i];
                    }
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
                const float r = 1.0f / sqrtf(ss / (float)p.D + p.eps);
                const float m = r * r * gx / (float)p.D;  // mean(g h) r
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

// f(lanes, elements, units, layout) of the instance for these sizes: E = 4 where
// pairs come in groups of four (rot_dim a multiple of 8), else pair by pair.
template <class F>
hipError_t by_shape(int D, int rot, bool inter, F&& f) {
    auto with = [&](auto L, auto E, auto NU) {
        return inter ? f(L, E, NU, std::true_type{}) : f(L, E, NU, std::false_type{});
    };
    std::integral_constant<int, 1> i1;
    std::integral_constant<int, 2> i2;
    std::integral_constant<int, 4> i4;
    if (rot % 8 != 0) return with(std::integral_constant<int, 64>{}, i1, i2);
    if (D <= 64) return with(std::integral_constant<int, 8>{}, i4, i1);
    if (D <= 128) return with(std::integral_constant<int, 16>{}, i4, i1);
    return with(std::integral_constant<int, 32>{}, i4, i1);
}

template <class T>
hipError_t forward(RopeArgs a, bool inter, hipStream_t st) {
    return by_shape(a.D, a.rot, inter, [&](auto L, auto E, auto NU, auto INTER) {
        constexpr int groups = 256 / decltype(L)::value;
        const int H = a.Hq + a.Hk + a.Hv;
        // tokens a workgroup: as many as leave eight workgroups for every compute
        // unit (a workgroup's first reads and angles take about as long as the
        // reads of three of its rounds); with small heads until its items fill its lanes, while every
        // compute unit has a workgroup
        a.tb = 1;
        const int wgs = getenv("RW") ? atoi(getenv("RW")) : 2048;
        while (2 * a.tb * (a.rot / 2) <= kRopeTrig &&
               cdiv_i(a.T, 2 * a.tb) >= (a.tb * H < groups ? 256 : wgs))
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
    return by_shape(a.D, a.rot, inter, [&](auto L, auto E, auto NU, auto INTER) {
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
