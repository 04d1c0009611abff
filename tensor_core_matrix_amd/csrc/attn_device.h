// What the attention kernels over a paged cache share on the device: 16-bit operands and the
// two parts of a probability, loads of rows, and exchanges between lane groups.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "tcm_device.h"

namespace tcm {

namespace {

constexpr float kNegInf = -__builtin_inff();

// kLift: what probabilities are multiplied by on their way into the second product, whose
// result is divided by it where the waves' parts meet.  They are at most 1, and fp16 ends at
// 2^-24: as they are, thousands of keys 2^-25 below the largest would vanish from the
// product and count in the sum.  bf16 has fp32's exponents.
// parts: two probabilities, times kLift, as upper parts (cut off) and lower parts (rounded).
// The upper one is cut from a number a little smaller, so that the lower one is
// never zero, and both are positive: an infinite value times them is infinite.  (fp16
// ends before it for probabilities below 2^-26.)
template <class T> struct Half16;
template <> struct Half16<__bf16> {
    static constexpr float kLift = 1.0f, kBelow = 0x1.fffff8p-1f;  // 1 - 2^-22
    typedef bf16x8_t x8;
    __device__ static __forceinline__ void parts(float e0, float e1, uint32_t& upper, uint32_t& lower) {
        const uint32_t b0 = __float_as_uint(e0 * kBelow), b1 = __float_as_uint(e1 * kBelow);
        upper = __builtin_amdgcn_perm(b1, b0, 0x07060302);
        typedef __bf16 pair __attribute__((ext_vector_type(2)));
        const pair r = {(__bf16)(e0 - __uint_as_float(b0 & 0xffff0000u)), (__bf16)(e1 - __uint_as_float(b1 & 0xffff0000u))};
        lower = __builtin_bit_cast(uint32_t, r);
    }
    __device__ static __forceinline__ f32x4_t mma(x8 a, x8 b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    __device__ static __forceinline__ uint32_t from_fp8(uint32_t w, bool hi) {
        return __builtin_bit_cast(uint32_t, hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    }
};
template <> struct Half16<_Float16> {
    static constexpr float kLift = 32768.0f, kBelow = 32768.0f - 2.0f;  // (1 - 2^-14)
    typedef f16x8_t x8;
    __device__ static __forceinline__ void parts(float e0, float e1, uint32_t& upper, uint32_t& lower) {
        const auto u = __builtin_amdgcn_cvt_pkrtz(e0 * kBelow, e1 * kBelow);
        upper = __builtin_bit_cast(uint32_t, u);
        const f16x2_t r = {(_Float16)fmaf(e0, kLift, -(float)u[0]), (_Float16)fmaf(e1, kLift, -(float)u[1])};
        lower = __builtin_bit_cast(uint32_t, r);
    }
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
        const v_t v = __builtin_nontemporal_load((const v_t*)(p + i * B));
#pragma unroll
        for (int j = 0; j < B / 4; ++j) w[i * (B / 4) + j] = v[j];
    }
}

// An int32 at a wave-uniform address that no kernel of the call writes, read
// through the scalar cache: its wait is apart from the vector loads', so a page's
// number can be looked up while a tile is on its way.
__device__ __forceinline__ int scalar_int(const int32_t* p) {
    return *(const __attribute__((address_space(4))) int32_t*)p;
}

// The larger of x and of lane l ^ 16's, and then of lane l ^ 32's, by register
// exchanges between rows of 16 and halves of the wave (no trip through LDS).
__device__ __forceinline__ float max_over_groups(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

}  // namespace

}  // namespace tcm
