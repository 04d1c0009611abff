// s = x + r, y = w s / sqrt(mean(s^2) + eps) and its gradients, row by row.
//
// Bound by memory: x, r, s and y pass once each.  A row lies in the registers of the
// lanes that share it (pieces of 8 elements, 16 bytes of each operand, dealt to the lanes in turn), so
// that the mean is known before anything is written and a row may be written onto itself.
#include "step_internal.h"
#include "tcm_device.h"

namespace tcm {

namespace {

constexpr int kNormGroups = 1 << 21;  // workgroups of a launch, at most

template <class T> struct Piece;
template <> struct Piece<__bf16> { typedef bf16x8_t type; };
template <> struct Piece<_Float16> { typedef f16x8_t type; };

template <class T>
__device__ __forceinline__ void load8(const T* p, float* v) {
    const typename Piece<T>::type x = *(const typename Piece<T>::type*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)x[i];
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float* v) {
    typename Piece<T>::type x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = convert_out<T>(v[i]);
    *(typename Piece<T>::type*)p = x;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
    *(f32x4_t*)p = (f32x4_t){v[0], v[1], v[2], v[3]};
    *(f32x4_t*)(p + 4) = (f32x4_t){v[4], v[5], v[6], v[7]};
}
// 8 weights of either type, or ones
template <class T>
__device__ __forceinline__ void load_weight(const NormArgs& a, int d, float* v) {
    if (!a.w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    } else if (a.w_f32) {
        const f32x4_t x = *(const f32x4_t*)((const float*)a.w + d), y = *(const f32x4_t*)((const float*)a.w + d + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < 4 ? x[i] : y[i - 4];
    } else {
        load8<T>((const T*)a.w + d, v);
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// over the 4 lanes of a quad
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, dpp<0xB1>(x));
    return fmaxf(x, dpp<0x4E>(x));
}
__device__ __forceinline__ float wave_sum(float x) {
    x += dpp<0xB1>(x);
    x += dpp<0x4E>(x);
    x += dpp<0x141>(x);
    x += dpp<0x140>(x);
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}
// Sum over the L lanes that share a row; `red` has a place for each wave of the workgroup.  A wave may
// be a sum ahead of the others, so sums take two such arrays in turn.
template <int L>
__device__ __forceinline__ float row_sum(float x, float* red) {
    x = wave_sum(x);
    if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0.0f;
#pragma unroll
        for (int i = 0; i < L / 64; ++i) x += red[i];
    }
    return x;
}

// 1 / sqrt(x): the hardware's approximation (1 ulp) and one Newton step.  The instruction takes subnormal numbers for
// zero, so those go through it 2^24 times as large.
__device__ __forceinline__ float inv_sqrt(float x) {
    const bool small = x < 0x1p-126f;
    const float y = small ? x * 0x1p24f : x;
    const float r = __builtin_amdgcn_rsqf(y);
    const float e = 0.5f - 0.5f * y * r * r;
    // (zero, infinite and NaN x have no step)
    return (e == e ? fmaf(r, e, r) : r) * (small ? 0x1p12f : 1.0f);
}

// The 8 elements of this lane, of 32 that four lanes share, in E4M3, and their scale
__device__ __forceinline__ void store_mx(uint8_t* out, uint8_t* scale, const float* y, bool first) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[i]) < __builtin_inff() ? fabsf(y[i]) : 0.0f);
    top = quad_max(top);
    // 448 = 0.875 * 2^9
    int e = __builtin_amdgcn_frexp_expf(top) - 9 + (__builtin_amdgcn_frexp_mantf(top) > 0.875f);
    e = top == 0.0f || e < -127 ? -127 : e;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = fabsf(y[i]) < __builtin_inff() ? __builtin_ldexpf(y[i], -e) : __builtin_nanf("");
    i32x2_t v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
        v[i] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], lo, true);
    }
    *(i32x2_t*)out = v;
    if (first) *scale = (uint8_t)(e + 127);
}

// L lanes a row, P pieces a lane (L * P * 8 elements at most); 256 lanes, or L of them.
template <class T, NormOut OUT, int L, int P>
__global__ __launch_bounds__(L > 256 ? L : 256) void norm_kernel(NormArgs a) {
    constexpr int ROWS = L > 256 ? 1 : 256 / L;
    __shared__ float red[2][L / 64];
    const int lane = threadIdx.x % L;
    int turn = 0;
    // (a launch ends at 2^32 threads, so workgroups go on where rows are left; those of more
    // than a wave take one row at a time)
    const int64_t first = (int64_t)blockIdx.x * ROWS + threadIdx.x / L;
    for (int64_t row = first; row < a.T; row += (int64_t)gridDim.x * ROWS, turn ^= 1) {
        const T* x = (const T*)a.x + row * a.ldx;
        const T* r = (const T*)a.r + row * a.ldr;
        float v[P][8];
        float sq = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int d = (p * L + lane) * 8;
            if (d < a.D) {
                load8<T>(x + d, v[p]);
                if (a.r) {
                    float u[8];
                    load8<T>(r + d, u);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[p][i] += u[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sq = fmaf(v[p][i], v[p][i], sq);
            }
        }
        const float f = inv_sqrt(row_sum<L>(sq, red[turn]) * a.inv_d + a.eps);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int d = (p * L + lane) * 8;
            if (d >= a.D) continue;
            if (a.sum) store8<T>((T*)a.sum + row * a.lds + d, v[p]);
            float w[8];
            load_weight<T>(a, d, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= v[p][i] * f;
            if constexpr (OUT == kNormHalf) {
                store8<T>((T*)a.out + row * a.ldo + d, w);
            } else if constexpr (OUT == kNormF32) {
                store8((float*)a.out + row * a.ldo + d, w);
            } else {
                const int64_t at = row * a.D + d;
                store_mx((uint8_t*)a.out + at, a.scale + at / 32, w, lane % 4 == 0);
            }
        }
    }
}

// A workgroup takes rows blockIdx.x, + gridDim.x, .. with L lanes each; a lane's columns are the same in every row,
// so it sums their weight gradients in registers.  Where there is room (P < 4) the next row is on its way while
// this one is worked on, and the weights stay too: of the next row nobody has written anything, also where dX is an
// operand, since rows are one workgroup's.  8192 x 4096 with dsum, bf16: 50 us, 5.4 TB/s, and 4.7 for the sum of
// the partial sums (75 and 10 with loads when they are needed and 64 workgroups for the sum).
template <class T, int L, int P, bool DW, bool R>
__global__ __launch_bounds__(L) void norm_bwd_kernel(NormArgs a) {
    typedef typename Piece<T>::type x8;
    constexpr bool AHEAD = P < 4;
    __shared__ float red[2][2][L / 64];
    const int lane = threadIdx.x;
    float dw[P][8], ws[AHEAD ? P : 1][8];
    struct Row {
        x8 v[P], g[P], u[P];
    };
    // (lanes past the end read the row's beginning; no load is under a condition, for exact waits)
    auto load = [&](Row& t, int64_t row) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int d = (p * L + lane) * 8 < a.D ? (p * L + lane) * 8 : 0;
            t.v[p] = *(const x8*)((const T*)a.x + row * a.ldx + d);
            t.g[p] = *(const x8*)((const T*)a.dy + row * a.lddy + d);
            if constexpr (R && AHEAD) t.u[p] = *(const x8*)((const T*)a.r + row * a.ldr + d);
        }
    };
    Row now, next;
    load(now, blockIdx.x);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if constexpr (AHEAD) load_weight<T>(a, (p * L + lane) * 8 < a.D ? (p * L + lane) * 8 : 0, ws[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[p][i] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const int64_t then = row + gridDim.x < a.T ? row + gridDim.x : row;
        if constexpr (AHEAD) load(next, then);
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if ((p * L + lane) * 8 < a.D) {
                float w[8];
                if constexpr (!AHEAD) load_weight<T>(a, (p * L + lane) * 8, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = (float)now.v[p][i];
                    sq = fmaf(v, v, sq);
                    dot = fmaf((float)now.g[p][i] * (AHEAD ? ws[p][i] : w[i]), v, dot);
                }
            }
        }
        // (two sets of places: a wave ahead by a row does not overwrite what others still read)
        sq = wave_sum(sq);
        dot = wave_sum(dot);
        if constexpr (L > 64) {
            if ((lane & 63) == 0) red[turn][0][lane >> 6] = sq, red[turn][1][lane >> 6] = dot;
            barrier_lds();  // (does not wait for the next row)
            sq = dot = 0.0f;
#pragma unroll
            for (int i = 0; i < L / 64; ++i) sq += red[turn][0][i], dot += red[turn][1][i];
        }
        const float f = inv_sqrt(sq * a.inv_d + a.eps);
        const float m = dot * f * a.inv_d;  // mean(g h)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int d = (p * L + lane) * 8;
            if (d >= a.D) continue;
            float w[8], o[8];
            if constexpr (!AHEAD) load_weight<T>(a, d, w);
            x8 u = {};
            if constexpr (R) u = AHEAD ? now.u[p] : *(const x8*)((const T*)a.r + row * a.ldr + d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float h = (float)now.v[p][i] * f, g = (float)now.g[p][i];
                if constexpr (DW) dw[p][i] = fmaf(g, h, dw[p][i]);
                o[i] = f * (g * (AHEAD ? ws[p][i] : w[i]) - h * m);
                if constexpr (R) o[i] += (float)u[i];
            }
            store8<T>((T*)a.out + row * a.ldo + d, o);
        }
        if constexpr (AHEAD) now = next;
        else load(now, then);
    }
    if constexpr (DW) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int d = (p * L + lane) * 8;
            if (d < a.D) store8(a.partial + (int64_t)blockIdx.x * a.D + d, dw[p]);
        }
    }
}

// The sum of the partial weight gradients of 16 columns: 4 lanes x 4 columns, 64 rows at a time, in a fixed order.
__global__ __launch_bounds__(256) void norm_dw_kernel(NormArgs a) {
    __shared__ __attribute__((aligned(16))) float part[4][16];
    const int c = threadIdx.x % 4 * 4, d = blockIdx.x * 16 + c;
    f32x4_t s = {};
    if (d < a.D) {
#pragma unroll 4
        for (int i = threadIdx.x / 4; i < a.groups; i += 64) s += *(const f32x4_t*)(a.partial + (int64_t)i * a.D + d);
    }
#pragma unroll
    for (int x = 4; x < 64; x *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += __shfl_xor(s[i], x);
    if (threadIdx.x % 64 < 4) *(f32x4_t*)&part[threadIdx.x / 64][c] = s;
    __syncthreads();
    const int mine = blockIdx.x * 16 + threadIdx.x;
    if (threadIdx.x < 16 && mine < a.D)
        a.dw[mine] = part[0][threadIdx.x] + part[1][threadIdx.x] + part[2][threadIdx.x] + part[3][threadIdx.x];
}

template <class T, NormOut OUT, int L, int P>
hipError_t run(const NormArgs& a, hipStream_t st) {
    constexpr int ROWS = L > 256 ? 1 : 256 / L;
    const int groups = min((a.T + ROWS - 1) / ROWS, kNormGroups);
    hipLaunchKernelGGL((norm_kernel<T, OUT, L, P>), dim3(groups), dim3(L > 256 ? L : 256), 0, st, a);
    return hipGetLastError();
}

template <class T, NormOut OUT>
hipError_t by_dim(const NormArgs& a, hipStream_t st) {
    if (a.D <= 512) return run<T, OUT, 64, 1>(a, st);
    if (a.D <= 2048) return run<T, OUT, 256, 1>(a, st);
    if (a.D <= 4096) return run<T, OUT, 256, 2>(a, st);
    if (a.D <= 8192) return run<T, OUT, 1024, 1>(a, st);
    return run<T, OUT, 1024, 4>(a, st);
}

template <class T>
hipError_t by_out(const NormArgs& a, NormOut out, hipStream_t st) {
    if (out == kNormHalf) return by_dim<T, kNormHalf>(a, st);
    return out == kNormF32 ? by_dim<T, kNormF32>(a, st) : by_dim<T, kNormMx>(a, st);
}

template <class T, int L, int P>
hipError_t run_bwd(const NormArgs& a, hipStream_t st) {
    const auto kernel = a.dw ? a.r ? norm_bwd_kernel<T, L, P, true, true> : norm_bwd_kernel<T, L, P, true, false>
                             : a.r ? norm_bwd_kernel<T, L, P, false, true> : norm_bwd_kernel<T, L, P, false, false>;
    hipLaunchKernelGGL(kernel, dim3(a.groups), dim3(L), 0, st, a);
    return hipGetLastError();
}

template <class T>
hipError_t bwd_by_dim(const NormArgs& a, hipStream_t st) {
    if (a.D <= 512) return run_bwd<T, 64, 1>(a, st);
    if (a.D <= 2048) return run_bwd<T, 256, 1>(a, st);
    if (a.D <= 4096) return run_bwd<T, 256, 2>(a, st);
    if (a.D <= 8192) return run_bwd<T, 1024, 1>(a, st);
    return run_bwd<T, 1024, 4>(a, st);
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs& a, int32_t dtype, NormOut out, hipStream_t st) {
    return dtype == 1 ? by_out<__bf16>(a, out, st) : by_out<_Float16>(a, out, st);
}

hipError_t launch_add_rms_norm_bwd(const NormArgs& a, int32_t dtype, hipStream_t st) {
    if (a.groups > 0) {
        const hipError_t e = dtype == 1 ? bwd_by_dim<__bf16>(a, st) : bwd_by_dim<_Float16>(a, st);
        if (e != hipSuccess) return e;
    }
    if (!a.dw) return hipSuccess;
    hipLaunchKernelGGL(norm_dw_kernel, dim3((a.D + 15) / 16), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace tcm
