// Low-rank adapters beside a product: what one wave adds to its accumulators.
//
// A row i of adapter a adds s_a (X[i] A_a^T) B_a^T.  The inner product is in
// memory (t, fp32, from lora_shrink_kernel); the second product runs on the
// matrix cores with the 16-row block's t as one operand and 16 rows of B_a as the
// other.  t keeps more than 16 bits through it as the sum of two 16-bit values:
// a 32-deep product holds 16 ranks twice, the upper halves of t in inner
// positions 0..15 and what they leave in 16..31, against the same 16 columns
// of B_a.  (One rounded t would add an error of the size of the output's own
// rounding where the adapter is as large as the projection; the second half
// costs nothing below rank 32 and little above it.)
//
// A block is multiplied once for every adapter that its 16 rows name, and only
// the rows that name it take the result: a row never sees another adapter's
// values, not even as 0 times infinity.
#pragma once

#include "layer_internal.h"
#include "tcm_device.h"

namespace tcm {

template <class T> struct LoraMma;
template <> struct LoraMma<__bf16> {
    typedef bf16x8_t x8;
    __device__ static __forceinline__ f32x4_t mma(x8 a, x8 b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct LoraMma<_Float16> {
    typedef f16x8_t x8;
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

// The t operand of ranks r0 .. r0 + 15 of the block's rows: lane l holds row
// l % 16, ranks r0 + 8 (g % 2) + 0..7 of the upper (g < 2) or lower half, g = l / 16.
// Lanes whose row is not `mine` get zeros (their t was never written).
template <class T>
__device__ __forceinline__ typename LoraMma<T>::x8 lora_t(const LoraArgs& p, int m, int r0, int g4,
                                                          bool mine) {
    typedef typename LoraMma<T>::x8 x8;
    const int r = r0 + 8 * (g4 & 1);
    x8 f = {};
    if (mine && r < p.R) {
        const float* t = p.t + (int64_t)m * p.R + r;
        f32x4_t a = *(const f32x4_t*)t, b = *(const f32x4_t*)(t + 4);
        for (int s = 1; s < p.ksplit; ++s) {
            const float* ts = t + (int64_t)s * p.M * p.R;
            a += *(const f32x4_t*)ts;
            b += *(const f32x4_t*)(ts + 4);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = j < 4 ? a[j & 3] : b[j & 3];
            const T hi = convert_out<T>(v);
            const float rest = v - (float)hi;
            // (where the upper half is infinite or NaN it says all)
            f[j] = g4 < 2 ? hi : rest == rest ? convert_out<T>(rest) : (T)0.0f;
        }
    }
    return f;
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

}  // namespace tcm
