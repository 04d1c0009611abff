// Low-rank adapters beside a product: what one wave adds to its accumulators.
//
// A row i of adapter a adds s_a (X[i] A_a^T) B_a^T.  The inner product is in
// memory (t, fp32, from lora_shrink_kernel); the second product runs on the
// matrix cores with the 16-row block's t as one operand and 16 rows of B_a as the
// other.  t keeps more than 16 bits through it as the sum of two 16-bit values:
// a 32-deep product holds 16 ranks twice, the upper halves of t in inner
// positions 0..15 and what they leave in 16..31, against the same 16 columns
// of B_a.  (One rounded t would add an error of the size of the output's own
// rounding where the adapter is as large as the projection.  The second half costs
// nothing up to rank 16, whose product is 32 deep anyway, and from there twice the
// products, which are few beside the projection's.)  For fp32 outputs of bf16
// operands a second product adds what the two halves leave.
//
// A row's 16 values are multiplied by a power of two first, which brings the largest of
// them into [2^14, 2^15), and the product by its inverse: fp16 ends at 65504, and below
// 2^-14 it has fewer digits.  So each step's product is taken by itself and added in fp32.
//
// A block is multiplied once for every adapter that its 16 rows name, and only
// the rows that name it take the result: a row never sees another adapter's
// values, not even as 0 times infinity.
#pragma once

#include "layer_internal.h"
#include "tcm_device.h"

namespace tcm {

// cut: x in the type, cut off a little nearer zero, so that what it leaves is never zero and
// has x's sign: an infinite element of B_a then gives its rows infinities, not NaN.
template <class T> struct LoraMma;
template <> struct LoraMma<__bf16> {
    typedef bf16x8_t x8;
    __device__ static __forceinline__ __bf16 cut(float x) {
        const uint32_t b = __float_as_uint(x * 0x1.fffff8p-1f);  // 1 - 2^-22
        return __builtin_bit_cast(__bf16, (uint16_t)(b >> 16));
    }
    __device__ static __forceinline__ f32x4_t mma(x8 a, x8 b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct LoraMma<_Float16> {
    typedef f16x8_t x8;
    __device__ static __forceinline__ _Float16 cut(float x) {
        return (_Float16)__builtin_amdgcn_cvt_pkrtz(x * 0x1.fff8p-1f, 0.0f)[0];  // 1 - 2^-14
    }
    __device__ static __forceinline__ f32x4_t mma(x8 a, x8 b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// Adapter of row m0 + l % 16 for lane l; -1: none (or no such row)
__device__ __forceinline__ int lora_row(const LoraArgs& p, int m0, int r16) {
    const int m = m0 + r16;
    const int a = m < p.M && p.L > 0 ? p.rows[m] : -1;
    return (uint32_t)a < (uint32_t)p.L ? a : -1;
}

__device__ __forceinline__ int lora_rank(const LoraArgs& p, int a) {
    const int r = p.ranks ? p.ranks[a] : p.R;
    return min(max(r, 0), p.R);
}

// t of row m, ranks r .. r + 7: the parts of K summed, four reads of them under way
// at a time
typedef float f32x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f32x8 lora_t8(const LoraArgs& p, int m, int r) {
    const float* t = p.t + (int64_t)m * p.R + r;
    f32x4_t a = {}, b = {};
    for (int s = 0; s < p.ksplit; s += 4) {
        f32x4_t u[4], v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (x == 0 || s + x < p.ksplit) {
                const float* ts = t + (int64_t)(s + x) * p.M * p.R;
                u[x] = *(const f32x4_t*)ts;
                v[x] = *(const f32x4_t*)(ts + 4);
            } else {
                u[x] = v[x] = (f32x4_t){};
            }
#pragma unroll
        for (int x = 0; x < 4; ++x) a += u[x], b += v[x];
    }
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The t operand of ranks r0 .. r0 + 15 of the block's rows: lane l holds row
// l % 16, ranks r0 + 8 (g % 2) + 0..7 of the upper (g < 2) or lower half, g = l / 16.
// Lanes whose row is not `mine` get zeros (their t was never written).  rest: what
// the two halves leave, half of it in each (FULL).  up: what the row's products are
// multiplied by.
template <class T> struct LoraT {
    typename LoraMma<T>::x8 f, rest;
    float up;
};
template <class T, bool FULL>
__device__ __forceinline__ LoraT<T> lora_t(const LoraArgs& p, int m, int r0, int g4, bool mine) {
    const int r = r0 + 8 * (g4 & 1);
    f32x8 t = {};
    if (mine && r < p.R) t = lora_t8(p, m, r);
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(t[j]));
    const auto both = __builtin_amdgcn_permlane16_swap(__float_as_uint(top), __float_as_uint(top), false, false);
    top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1]));
    // 2^k and 2^-k, both normal; an infinite value counts as the largest finite one
    const int k = min(14 + 127 - (int)(__float_as_uint(top) >> 23), 126);
    const float down = __uint_as_float((uint32_t)(127 + k) << 23);
    LoraT<T> o;
    o.up = __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = t[j] * down;
        const T hi = LoraMma<T>::cut(x);
        const float rest = x - (float)hi;
        // (an infinite or NaN upper half, which is t itself, says all)
        const T lo = rest != rest ? (T)0.0f : FULL ? LoraMma<T>::cut(rest) : convert_out<T>(rest);
        o.f[j] = g4 < 2 ? hi : lo;
        if constexpr (FULL) {
            const float last = rest - (float)lo;
            o.rest[j] = last == last ? convert_out<T>(0.5f * last) : (T)0.0f;
        }
    }
    return o;
}

// The B operand: row n of B_a, the same ranks; zeros from the adapter's rank on.
template <class T>
__device__ __forceinline__ typename LoraMma<T>::x8 lora_b(const LoraArgs& p, int a, int rank, int n,
                                                          int r0, int g4) {
    typedef typename LoraMma<T>::x8 x8;
    const int r = r0 + 8 * (g4 & 1);
    x8 f = {};
    if (r < rank) {
        f = *(const x8*)((const T*)p.B + ((int64_t)a * p.N + min(n, p.N - 1)) * p.R + r);
        if (r + 8 > rank) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = r + j < rank ? f[j] : (T)0.0f;
        }
    }
    return f;
}

// The adapters' part of a block of 16 NI rows from m0 and 16 NJ columns from n0,
// added to acc[i][j] (lane l: row 16 i + l % 16, columns 16 j + 4 (l / 16) ..), block of
// rows by block.  A block that names one or two adapters (the rule where requests
// bring whole prompts) takes the matrix cores, once for each; one that names more
// (a decode batch: nearly every row its own) is left to its lanes, each of which
// adds up its own columns of its own row's adapter in fp32, all of a block's reads
// under way together: adapter by adapter, 128 rows with 64 adapters (4096 x 4096,
// rank 16) take 71 us, this way 29 (16 without adapters; 78 at rank 64, whose every 8
// ranks wait for their reads).
template <class T, bool FULL, int NI, int NJ>
__device__ __forceinline__ void lora_add(const LoraArgs& p, f32x4_t (&acc)[NI][NJ], int m0, int n0) {
    typedef LoraMma<T> O;
    typedef typename O::x8 x8;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
    int ids[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) ids[i] = lora_row(p, m0 + 16 * i, r16);
    // the wave's whole stretch of rows has one adapter: its operands are read once
    const int one = __builtin_amdgcn_readfirstlane(ids[0]);
    bool same = one >= 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) same = same && ids[i] == one;
    if (__ballot(!same) == 0) {
        const int rank = lora_rank(p, one);
        for (int r0 = 0; r0 < rank; r0 += 16) {
            x8 b[NJ];
            LoraT<T> t[NI];
#pragma unroll
            for (int j = 0; j < NJ; ++j) b[j] = lora_b<T>(p, one, rank, n0 + 16 * j + r16, r0, g4);
#pragma unroll
            for (int i = 0; i < NI; ++i) t[i] = lora_t<T, FULL>(p, m0 + 16 * i + r16, r0, g4, true);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    f32x4_t d = O::mma(b[j], t[i].f, (f32x4_t){});
                    if constexpr (FULL) d = O::mma(b[j], t[i].rest, d);
                    acc[i][j] += d * t[i].up;
                }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int m = m0 + 16 * i + r16, id = ids[i];
        uint32_t left = (uint32_t)__ballot(id >= 0) & 0xffffu;
        if (!left) continue;
        const int first = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
        const uint32_t others = left & ~(uint32_t)__ballot(id == first);
        const int second = others ? __builtin_amdgcn_readlane(id, __builtin_ctz(others)) : first;
        if ((others & ~(uint32_t)__ballot(id == second)) == 0) {
            while (left) {
                const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
                left &= ~(uint32_t)__ballot(id == a);
                const int rank = lora_rank(p, a);
                for (int r0 = 0; r0 < rank; r0 += 16) {
                    x8 b[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) b[j] = lora_b<T>(p, a, rank, n0 + 16 * j + r16, r0, g4);
                    const LoraT<T> t = lora_t<T, FULL>(p, m, r0, g4, id == a);
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        f32x4_t d = O::mma(b[j], t.f, (f32x4_t){});
                        if constexpr (FULL) d = O::mma(b[j], t.rest, d);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][e] += id == a ? d[e] * t.up : 0.0f;
                    }
                }
            }
            continue;
        }
        const int rank = id >= 0 ? lora_rank(p, id) : 0;
        const T* const brow = (const T*)p.B + (int64_t)max(id, 0) * p.N * p.R;
        for (int r = 0; r < p.R; r += 8) {
            if (__ballot(r < rank) == 0) break;
            if (r >= rank) continue;
            const f32x8 t = lora_t8(p, m, r);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                x8 b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    b[e] = *(const x8*)(brow + (int64_t)min(n0 + 16 * j + 4 * g4 + e, p.N - 1) * p.R + r);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float s = 0.0f;
#pragma unroll
                    for (int x = 0; x < 8; ++x) s += r + x < rank ? t[x] * (float)b[e][x] : 0.0f;
                    acc[i][j][e] += s;
                }
            }
        }
    }
}

// The same for accumulators that leave few registers: always the matrix cores, block
// of rows by block and adapter by adapter, four columns' blocks at a time.
template <class T, bool FULL, int NI, int NJ>
__device__ __forceinline__ void lora_add_lean(const LoraArgs& p, f32x4_t (&acc)[NI][NJ], int m0, int n0) {
    typedef LoraMma<T> O;
    typedef typename O::x8 x8;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int id = lora_row(p, m0 + 16 * i, r16);
        uint32_t left = (uint32_t)__ballot(id >= 0) & 0xffffu;
        while (left) {
            const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
            left &= ~(uint32_t)__ballot(id == a);
            const int rank = lora_rank(p, a);
            for (int r0 = 0; r0 < rank; r0 += 16) {
                const LoraT<T> t = lora_t<T, FULL>(p, m0 + 16 * i + r16, r0, g4, id == a);
#pragma unroll
                for (int j0 = 0; j0 < NJ; j0 += 4) {
                    x8 b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = lora_b<T>(p, a, rank, n0 + 16 * (j0 + j) + r16, r0, g4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        f32x4_t d = O::mma(b[j], t.f, (f32x4_t){});
                        if constexpr (FULL) d = O::mma(b[j], t.rest, d);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j0 + j][e] += id == a ? d[e] * t.up : 0.0f;
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }
}

}  // namespace tcm
