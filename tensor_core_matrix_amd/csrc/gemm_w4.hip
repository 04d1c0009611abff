// Out = X W^T for few rows X and 4-bit weights W.
//
// Bound by memory: the weights pass once for each 64 rows of X.  A wave takes 16 NT columns
// (rows of W) and blocks of 128 values of K: a lane reads 16 bytes, 32 values of one
// row of W, so four lanes read 64 bytes of a row.  The products are 16 x 16 x 32, X the first
// operand and W the second:
//
//   Out (16 rows x 16 columns) += X (16 x 32) W^T (32 x 16)
//
// A product's 32 values have one scale a column, so they must be 32 values that follow each
// other; the four lanes that hold the 128 of a row trade their words (a transposition of
// 4 x 4 words by register exchanges between rows of lanes) and each gets 8 of every 32.
//
// The whole numbers 0 .. 15 are E4M3 bytes times 2^9 as they are -- below 8 the byte is
// subnormal, q 2^-9, and from 8 on it has exponent 1: (1 + (q - 8) / 8) 2^-6 -- so the
// conversion of E4M3 pairs gives both 16-bit types exactly.  The zero point is a second
// product with the same X and a constant -zero.  Sums of a group are fp32 and are multiplied
// by its scale in fp32.  E2M1 elements have a conversion of their own.
//
// The waves of a workgroup take K blocks in turn; their sums meet in LDS.
#include "step_internal.h"
#include "tcm_device.h"

namespace tcm {

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <class T> struct Half;
template <> struct Half<__bf16> {
    typedef bf16x8_t x8;
    __device__ static __forceinline__ f32x4_t mma(x8 a, x8 b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // bytes 0, 1 or 2, 3 of w, E4M3, times s
    template <bool HI>
    __device__ static __forceinline__ uint32_t from_fp8(uint32_t w, float s) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HI));
    }
    // the two E2M1 elements of byte B of w
    template <int B>
    __device__ static __forceinline__ uint32_t from_fp4(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, B));
    }
};
template <> struct Half<_Float16> {
    typedef f16x8_t x8;
    __device__ static __forceinline__ f32x4_t mma(x8 a, x8 b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    template <bool HI>
    __device__ static __forceinline__ uint32_t from_fp8(uint32_t w, float s) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, HI));
    }
    template <int B>
    __device__ static __forceinline__ uint32_t from_fp4(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, B));
    }
};

// Rows 0 .. 3 of 16 lanes hold a word each; w[i] becomes row i's in all of them.
__device__ __forceinline__ void spread(uint32_t x, uint32_t* w) {
    const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
    w[0] = b[0];
    w[1] = b[1];
    w[2] = c[0];
    w[3] = c[1];
}
// Word i of row g of 16 lanes changes places with word g of row i.
__device__ __forceinline__ void turn(u32x4_t& w) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = (u32x4_t){c[0], c[1], d[0], d[1]};
}

// 8 elements of a word, in order, as an operand
template <class T, bool E2M1>
__device__ __forceinline__ typename Half<T>::x8 expand(uint32_t w) {
    typedef Half<T> H;
    u32x4_t v;
    if constexpr (E2M1) {
        v = (u32x4_t){H::template from_fp4<0>(w), H::template from_fp4<1>(w), H::template from_fp4<2>(w),
                      H::template from_fp4<3>(w)};
    } else {
        const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
        const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400), hi = __builtin_amdgcn_perm(odd, even, 0x07030602);
        v = (u32x4_t){H::template from_fp8<false>(lo, 512.0f), H::template from_fp8<true>(lo, 512.0f),
                      H::template from_fp8<false>(hi, 512.0f), H::template from_fp8<true>(hi, 512.0f)};
    }
    return __builtin_bit_cast(typename H::x8, v);
}
template <class T>
__device__ __forceinline__ typename Half<T>::x8 splat(float x) {
    typename Half<T>::x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = convert_out<T>(x);
    return v;
}

constexpr int kWaves = 8;

// MT: products of 16 rows; NT: of 16 columns of a wave.
template <class T, class TO, bool E2M1, int MT, int NT>
__global__ __launch_bounds__(kWaves * 64) void w4_kernel(W4Args a) {
    typedef Half<T> H;
    typedef typename H::x8 x8;
    __shared__ __attribute__((aligned(16))) f32x4_t part[kWaves][MT * NT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT;
    const int chunks = a.K / 32;

    // this lane's rows of X and of W (past the last: the last, whose results nobody stores)
    const T* xr[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) xr[i] = (const T*)a.x + (int64_t)min(m0 + 16 * i + r16, a.M - 1) * a.ldx + 8 * g4;
    const uint8_t* wr[NT];
    int64_t sr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = min(n0 + 16 * j + r16, a.N - 1);
        wr[j] = a.w + (int64_t)n * (a.K / 2) + 16 * g4;
        sr[j] = (int64_t)n * a.groups;
    }

    struct Block {
        u32x4_t w[NT];
        uint32_t s[NT];  // scale, zero point << 16
        x8 x[MT][4];
    };
    auto load = [&](Block& t, int c0) {
        const int c = min(c0 + g4, chunks - 1);  // (chunks past the end are not used)
        const int g = E2M1 ? c : a.gshift >= 0 ? c >> a.gshift : c / a.gchunks;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            t.w[j] = __builtin_nontemporal_load((const u32x4_t*)(wr[j] + (int64_t)(c - g4) * 16));
            if constexpr (E2M1) {
                t.s[j] = ((const uint8_t*)a.scales)[sr[j] + g];
            } else {
                t.s[j] = ((const uint16_t*)a.scales)[sr[j] + g] | (a.zeros ? (uint32_t)a.zeros[sr[j] + g] : 8u) << 16;
            }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int k = min(c0 + y, chunks - 1) * 32;
#pragma unroll
            for (int i = 0; i < MT; ++i) t.x[i][y] = *(const x8*)(xr[i] + k);
        }
    };
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = (f32x4_t){};
    auto compute = [&](Block& t, int c0) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            uint32_t s[4];
            spread(t.s[j], s);
            turn(t.w[j]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                if (c0 + y >= chunks) break;
                const x8 b = expand<T, E2M1>(t.w[j][y]);
                float scale;
                x8 zero;
                if constexpr (E2M1) {
                    // 2^-127 is subnormal, and 255 stands for NaN
                    scale = __uint_as_float(s[y] == 0 ? 0x00400000u : s[y] == 255 ? 0x7fc00000u : s[y] << 23);
                } else {
                    scale = (float)__builtin_bit_cast(T, (uint16_t)s[y]);
                    zero = splat<T>(-(float)(s[y] >> 16));
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    f32x4_t p = H::mma(t.x[i][y], b, (f32x4_t){});
                    if constexpr (!E2M1) p = H::mma(t.x[i][y], zero, p);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(scale, p[r], acc[i][j][r]);
                }
            }
        }
    };
    int c = wave * 4;
    if (c < chunks) {
        Block p, q;
        load(p, c);
        for (;;) {
            const int d = c + kWaves * 4;
            if (d < chunks) load(q, d);
            compute(p, c);
            if (d >= chunks) break;
            c = d + kWaves * 4;
            if (c < chunks) load(p, c);
            compute(q, d);
            if (c >= chunks) break;
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    for (int t = wave; t < MT * NT; t += kWaves) {
        f32x4_t s = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += part[w][t][lane];
        const int n = n0 + t % NT * 16 + r16;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int m = m0 + t / NT * 16 + 4 * g4 + r;
            if (m < a.M && n < a.N) ((TO*)a.out)[m * a.ldo + n] = convert_out<TO>(s[r]);
        }
    }
}

template <class T, class TO, bool E2M1, int MT, int NT>
hipError_t run(const W4Args& a, hipStream_t st) {
    const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (a.M + 16 * MT - 1) / (16 * MT));
    hipLaunchKernelGGL((w4_kernel<T, TO, E2M1, MT, NT>), grid, dim3(kWaves * 64), 0, st, a);
    return hipGetLastError();
}

template <class T, class TO, bool E2M1>
hipError_t by_rows(const W4Args& a, hipStream_t st) {
    if (a.M <= 16) return run<T, TO, E2M1, 1, 1>(a, st);
    if (a.M <= 32) return run<T, TO, E2M1, 2, 2>(a, st);
    return run<T, TO, E2M1, 4, 2>(a, st);
}

template <class T>
hipError_t by_type(const W4Args& a, bool e2m1, bool out_f32, hipStream_t st) {
    if (e2m1) return out_f32 ? by_rows<T, float, true>(a, st) : by_rows<T, T, true>(a, st);
    return out_f32 ? by_rows<T, float, false>(a, st) : by_rows<T, T, false>(a, st);
}

}  // namespace

hipError_t launch_gemm_w4(const W4Args& a, int32_t dtype, bool e2m1, bool out_f32, int cus, hipStream_t st) {
    return dtype == 1 ? by_type<__bf16>(a, e2m1, out_f32, st) : by_type<_Float16>(a, e2m1, out_f32, st);
}

}  // namespace tcm
