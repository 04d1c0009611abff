// Out = X W^T for few rows X and 4-bit weights W.
//
// Bound by memory while X has few rows, since every 64 rows pass over the weights once; from about 40 rows on
// loads, unpacking (about 90 vector instructions a block of 16 x 128) and X's way through LDS take about the same
// time each.  Measured on an MI355X, weights as a rule not in a cache:
//
//   M   N      K     elements, group, type      us     weights and scales, TB/s
//   1   4096   4096  U4, 128, zeros, bf16       8.3    1.1  (most of it the call itself)
//   12  12288  4096  E2M1, 32, bf16             10.5   2.6
//   48  32003  4096  U4, 64, fp16 to fp32       28.5   2.4
//
// A wave takes 16 columns (rows of W) and blocks of 128 values of K: a lane reads 16 bytes, 32 values of one
// row of W, so four lanes read 64 bytes of a row, and a batch of 4 blocks that follow each other 256: whole
// lines, one after the other.  The products are 16 x 16 x 32, X the first operand and W the second:
//
//   Out (16 rows x 16 columns) += X (16 x 32) W^T (32 x 16)
//
// A product's 32 values have one scale a column, so they must be 32 values that follow each
// other; the four lanes that hold the 128 of a row trade their words (a transposition of
// 4 x 4 words by register exchanges between rows of lanes) and each gets 8 of every 32.
//
// The whole numbers 0 .. 15 are E4M3 bytes times 2^9 as they are -- below 8 the byte is subnormal, q 2^-9, and from
// 8 on it has exponent 1: (1 + (q - 8) / 8) 2^-6 -- so the conversion of E4M3 pairs gives both 16-bit types
// exactly.  Zero points are subtracted from elements of fp16, which have packed subtractions; for bf16, which has
// none, they are a second product with the same X and a constant -zero.  Sums of a group are fp32 and are
// multiplied by its scale in fp32.  E2M1 elements have a conversion of their own.
//
// What the loads need, found by leaving parts out (the call of 48 rows, 82 us at first):
//   - X in LDS, once for all waves of a workgroup, 42.  Read by each wave for itself it was the largest part: 66,
//     and 35 where all read the same address.
//   - No load under a condition: the compiler waits, where two ways meet, for what is certain on both.
//   - A lane's scales in one load a batch rather than one a block, 37.  So a lane's row of scales has to be
//     aligned; sizes where it is not (PER == 0) load one a block.
//   - Stages of X through registers, 35: copies straight into LDS, which the compiler does not count, made each wait
//     for W one for the copies behind it.
//   - Packed subtractions and one addition for each address in LDS, 29.  Now no part left out by itself gains more
//     than 2.
//
// Waves of a workgroup stand side by side, or take K in turn where N alone leaves compute units without work; their
// sums meet in LDS.
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

// 8 elements of a word, in order, as an operand; MINUS (fp16): less z, whole numbers both, which is exact
template <class T, bool E2M1, bool MINUS>
__device__ __forceinline__ typename Half<T>::x8 expand(uint32_t w, _Float16 z) {
    typedef Half<T> H;
    uint32_t v[4];
    if constexpr (E2M1) {
        v[0] = H::template from_fp4<0>(w);
        v[1] = H::template from_fp4<1>(w);
        v[2] = H::template from_fp4<2>(w);
        v[3] = H::template from_fp4<3>(w);
    } else {
        const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
        const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400), hi = __builtin_amdgcn_perm(odd, even, 0x07030602);
        v[0] = H::template from_fp8<false>(lo, 512.0f);
        v[1] = H::template from_fp8<true>(lo, 512.0f);
        v[2] = H::template from_fp8<false>(hi, 512.0f);
        v[3] = H::template from_fp8<true>(hi, 512.0f);
    }
    if constexpr (MINUS) {
        // (pair by pair: of a vector of eight the compiler makes single subtractions)
        const f16x2_t zz = {z, z};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, v[i]) - zz);
    }
    return __builtin_bit_cast(typename H::x8, (u32x4_t){v[0], v[1], v[2], v[3]});
}
template <class T>
__device__ __forceinline__ typename Half<T>::x8 splat(float x) {
    typename Half<T>::x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = convert_out<T>(x);
    return v;
}

// (as in the attention of drafted tokens: the resource may come out of vector registers)
__device__ __forceinline__ void copy16_to_lds_far(__amdgpu_buffer_rsrc_t r, void* lds_wave_base, uint32_t voffset) {
    const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds_wave_base;
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(at);
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voffset), "s"(r), "{m0}"(m0) : "memory");
}

// Waves of a workgroup, and blocks of 128 values that each has under way: a batch.  (More than 32 rows leave no
// room in LDS for a stage of more than 512 values; 16 waves on those took 28.5 us for the case above, 8 took 29.4.)
constexpr int waves_of(int MT) { return MT > 2 ? 16 : 8; }
constexpr int depth_of(int MT) { return MT > 2 ? 2 : 4; }
constexpr int kStageBytes = 64 * 1024;  // of LDS for X, twice

// MT: products of 16 rows.  PER: a scale is for 1, 2 or 4 chunks of 32 (4: or a multiple), K a multiple of 128 and
// the scales aligned to those of a block; 0: any of the rest. STAGED: X passes through LDS in stages of a batch of
// each wave; else it is there as a whole.
template <class T, class TO, bool E2M1, int MT, int PER, bool STAGED>
__global__ __launch_bounds__(waves_of(MT) * 64, waves_of(MT) / 4) void w4_kernel(W4Args a) {
    constexpr int kWaves = waves_of(MT), kDepth = depth_of(MT);
    typedef Half<T> H;
    typedef typename H::x8 x8;
    constexpr bool EXACT = !E2M1 && std::is_same<T, _Float16>::value;  // zero points leave the elements
    extern __shared__ __attribute__((aligned(1024))) char lds[];       // X; in the end the waves' sums
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & (a.wn - 1), wk = wave / a.wn, WK = kWaves / a.wn;
    const int r16 = lane & 15, g4 = lane >> 4;
    const int n0 = (blockIdx.x * a.wn + wn) * 16, m0 = blockIdx.y * a.rows;
    const int rows = min(a.rows, a.M - m0);
    const int chunks = a.K / 32, blocks = (chunks + 3) / 4;

    // this lane's row of W (past the last: the last, whose results nobody stores)
    const int n = min(n0 + r16, a.N - 1);
    const u32x4_t* const wr = (const u32x4_t*)(a.w + (int64_t)n * (a.K / 2));
    const int64_t sr = (int64_t)n * a.groups;
    const uint8_t* const zeros = a.zeros ? a.zeros : (const uint8_t*)a.scales;
    auto load = [&](int block) { return wr[min(4 * block + g4, chunks - 1)]; };  // (chunks past the end are not used)

    // Scales and zero points.  PER > 0: lane row g4 holds those of a batch's block g4.  PER == 0: of chunk g4 of
    // each block.  Raw: put together where they are used, since that waits for them.
    constexpr int SB = E2M1 ? 1 : 2, NS = PER > 0 ? 4 / PER : 1;
    struct Scales {
        uint32_t s[PER > 0 ? (NS * SB + 3) / 4 : kDepth];
        uint32_t z[PER > 0 ? 1 : kDepth];
    };
    auto load_scales = [&](Scales& t, int block) {
        if constexpr (PER > 0) {
            const int b = min(block + g4, blocks - 1);
            const int g = PER < 4 ? b * NS : a.gshift >= 0 ? (4 * b) >> a.gshift : 4 * b / a.gchunks;
            __builtin_memcpy(t.s, __builtin_assume_aligned((const char*)a.scales + (sr + g) * SB, NS * SB), NS * SB);
            if constexpr (!E2M1) __builtin_memcpy(t.z, __builtin_assume_aligned(zeros + (a.zeros ? sr + g : 0), NS), NS);
        } else {
#pragma unroll
            for (int i = 0; i < kDepth; ++i) {
                const int c = min(4 * (block + i) + g4, chunks - 1);
                const int g = E2M1 ? c : a.gshift >= 0 ? c >> a.gshift : c / a.gchunks;
                t.s[i] = E2M1 ? ((const uint8_t*)a.scales)[sr + g] : ((const uint16_t*)a.scales)[sr + g];
                if constexpr (!E2M1) t.z[i] = zeros[a.zeros ? sr + g : 0];
            }
        }
    };

    // X: stages of a.kc values of every row.  A row's 16-byte piece c lies at c ^ (row % 16), so that the 16 rows
    // of an operand meet different banks.
    const int stage_bytes = (STAGED && MT > 2 ? 16 * MT : rows) * a.kc * 2, pieces = a.kc / 8;
    auto stage = [&](int s, int buffer) {
        // 64 pieces a copy, dealt to the waves; what lies past a row's end is zero
        for (int i = wave; i < rows * pieces / 64; i += kWaves) {
            const int row = i / (pieces / 64), c = i % (pieces / 64) * 64 + lane;
            copy16_to_lds_far(make_rsrc((const T*)a.x + (int64_t)(m0 + row) * a.ldx, (uint32_t)a.K * 2),
                              lds + buffer * stage_bytes + i * 1024, (uint32_t)(s * a.kc + (c ^ (row & 15)) * 8) * 2);
        }
    };
    // the same through registers, so that the compiler knows how many loads there are in its waits for W
    constexpr int XC = kStageBytes / 1024 / kWaves, XN = STAGED ? MT == 3 ? XC * 3 / 4 : XC : 1;
    u32x4_t xs[XN];
    auto stage_load = [&](int s) {
#pragma unroll
        for (int j = 0; j < XN; ++j) {
            const int i = min(wave + kWaves * j, rows * pieces / 64 - 1);
            const int row = i / (pieces / 64), c = i % (pieces / 64) * 64 + lane;
            const T* const from = (const T*)a.x + (int64_t)(m0 + row) * a.ldx;
            xs[j] = __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(from, (uint32_t)a.K * 2),
                                                          (uint32_t)(s * a.kc + (c ^ (row & 15)) * 8) * 2, 0, 0);
        }
    };
    auto stage_store = [&](int buffer) {
#pragma unroll
        for (int j = 0; j < XN; ++j) {
            const int i = wave + kWaves * j;
            if (i < rows * pieces / 64) *(u32x4_t*)(lds + buffer * stage_bytes + i * 1024 + lane * 16) = xs[j];
        }
    };
    // This lane's 16 bytes of chunk y of a block; of a row past the last, any.  KC: a.kc where it is always the
    // same, so that the rows' distance stands in the instructions.
    constexpr int KC = STAGED && MT > 2 ? 512 : 0;
    const char* xrow[KC > 0 ? 1 : MT];
    int piece[4];
    if constexpr (KC > 0) xrow[0] = lds + r16 * KC * 2;
    else
#pragma unroll
        for (int i = 0; i < MT; ++i) xrow[i] = lds + min(16 * i + r16, rows - 1) * a.kc * 2;
#pragma unroll
    for (int y = 0; y < 4; ++y) piece[y] = ((4 * y + g4) ^ r16) * 16;
    auto x_at = [&](int i, int y, int at) {
        if constexpr (KC > 0) return *(const x8*)(xrow[0] + (at + piece[y]) + i * 16 * KC * 2);
        else return *(const x8*)(xrow[i] + (at + piece[y]));
    };

    f32x4_t acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = (f32x4_t){};
    // at: the block's first byte in a row of X's stage; left: its chunks, 4 (but for a row's last block); s, z:
    // words that hold the scales and zero points, one a chunk (PER == 0) or those of the block
    auto compute = [&](u32x4_t w, const uint32_t* s, const uint32_t* z, int at, int left) {
        turn(w);
        f32x4_t p[MT];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (PER == 0 && y >= left) break;
            constexpr int EVERY = PER > 0 ? PER : 1;
            const int j = y / EVERY;
            uint32_t sy, zy;
            if constexpr (PER > 0) {
                sy = E2M1 ? s[0] >> (8 * j) & 0xff : s[j / 2] >> (16 * (j & 1)) & 0xffff;
                zy = z[0] >> (8 * j) & 0xff;
            } else {
                sy = s[y];
                zy = z[y];
            }
            const x8 b = expand<T, E2M1, EXACT>(w[y], EXACT ? (_Float16)(float)zy : (_Float16)0.0f);
            x8 x[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) x[i] = x_at(i, y, at);
            if (y % EVERY == 0)
#pragma unroll
                for (int i = 0; i < MT; ++i) p[i] = (f32x4_t){};
#pragma unroll
            for (int i = 0; i < MT; ++i) p[i] = H::mma(x[i], b, p[i]);
            if constexpr (!E2M1 && !EXACT) {
                const x8 zero = splat<T>(-(float)zy);
#pragma unroll
                for (int i = 0; i < MT; ++i) p[i] = H::mma(x[i], zero, p[i]);
            }
            if (y % EVERY == EVERY - 1) {
                float scale;
                // 2^-127 is subnormal, and 255 stands for NaN
                if constexpr (E2M1) scale = __uint_as_float(sy == 0 ? 0x00400000u : sy == 255 ? 0x7fc00000u : sy << 23);
                else scale = (float)__builtin_bit_cast(T, (uint16_t)sy);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][r] = fmaf(scale, p[i][r], acc[i][r]);
            }
        }
    };
    // A stage's batches are dealt to the waves that share K, `per` to each.  The loads of the next batch are always
    // under way, without conditions (past the end: the last chunk's again), so that the compiler knows which
    // ones a block has to wait for.
    const int stages = a.K > 0 ? (a.K + a.kc - 1) / a.kc : 0, per = a.kc / (128 * kDepth) / WK;
    auto batch = [&](int s, int j) { return (s * WK + wk) * per + j; };
    u32x4_t ring[kDepth];
    Scales next;
    if (stages > 0) {
        stage(0, 0);
        load_scales(next, batch(0, 0) * kDepth);
#pragma unroll
        for (int i = 0; i < kDepth; ++i) ring[i] = load(batch(0, 0) * kDepth + i);
    }
    wait_vmcnt<kDepth>();  // the copies are older than the loads of kDepth blocks
    for (int s = 0; s < stages; ++s) {
        barrier_lds();
        if constexpr (STAGED) stage_load(s + 1);
        for (int j = 0; j < per; ++j) {
            const Scales now = next;
            const int b = batch(s, j) * kDepth, then = (j + 1 < per ? batch(s, j + 1) : batch(s + 1, 0)) * kDepth;
            load_scales(next, then);
            uint32_t sw[kDepth][4], zw[kDepth][4];
            if constexpr (PER > 0) {
                uint32_t all[4];
#pragma unroll
                for (int i = 0; i < (NS * SB + 3) / 4; ++i) {
                    spread(now.s[i], all);
#pragma unroll
                    for (int k = 0; k < kDepth; ++k) sw[k][i] = all[k];
                }
                if constexpr (!E2M1) {
                    spread(a.zeros ? now.z[0] : 0x08080808, all);
#pragma unroll
                    for (int k = 0; k < kDepth; ++k) zw[k][0] = all[k];
                }
            }
            const int at = (s & 1) * stage_bytes + (wk * per + j) * kDepth * 256;
#pragma unroll
            for (int i = 0; i < kDepth; ++i) {
                const u32x4_t w = ring[i];
                ring[i] = load(then + i);
                const int left = chunks - 4 * (b + i);
                if (left > 0) {
                    if constexpr (PER == 0) {
                        spread(now.s[i], sw[i]);
                        if constexpr (!E2M1) spread(a.zeros ? now.z[i] : 8, zw[i]);
                    }
                    compute(w, sw[i], zw[i], at + i * 256, left);
                }
            }
        }
        if constexpr (STAGED) stage_store((s + 1) & 1);
    }
    // the parts of K, a product at a time
    barrier_lds();
    f32x4_t (*const part)[MT][64] = (f32x4_t (*)[MT][64])lds;
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int t = wave; t < a.wn * MT; t += kWaves) {
        const int from = t / MT, u = t % MT;
        f32x4_t s = part[from][u][lane];
        for (int w = 1; w < WK; ++w) s += part[from + w * a.wn][u][lane];
        const int c = (blockIdx.x * a.wn + from) * 16 + r16;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int m = u * 16 + 4 * g4 + r;
            if (m < rows && c < a.N) ((TO*)a.out)[(m0 + m) * a.ldo + c] = convert_out<TO>(s[r]);
        }
    }
}

template <class T, class TO, bool E2M1, int MT, bool STAGED>
hipError_t run(const W4Args& a, hipStream_t st) {
    constexpr int kWaves = waves_of(MT);
    const dim3 grid((a.N + 16 * a.wn - 1) / (16 * a.wn), (a.M + a.rows - 1) / a.rows), wg(kWaves * 64);
    const int x = (STAGED && MT > 2 ? 16 * MT : a.rows) * a.kc * 2 * (STAGED ? 2 : 1), sums = kWaves * MT * 1024;
    const int lds = x > sums ? x : sums;
    const auto aligned = [&](int n) {
        return a.K % 128 == 0 && (uintptr_t)a.scales % (n * (E2M1 ? 1 : 2)) == 0 && (uintptr_t)a.zeros % n == 0;
    };
    if constexpr (!E2M1) {
        if (a.gchunks % 4 == 0) {
            hipLaunchKernelGGL((w4_kernel<T, TO, false, MT, 4, STAGED>), grid, wg, lds, st, a);
            return hipGetLastError();
        }
        if (a.gchunks == 2 && aligned(2)) {
            hipLaunchKernelGGL((w4_kernel<T, TO, false, MT, 2, STAGED>), grid, wg, lds, st, a);
            return hipGetLastError();
        }
    }
    if (a.gchunks == 1 && aligned(4)) hipLaunchKernelGGL((w4_kernel<T, TO, E2M1, MT, 1, STAGED>), grid, wg, lds, st, a);
    else hipLaunchKernelGGL((w4_kernel<T, TO, E2M1, MT, 0, STAGED>), grid, wg, lds, st, a);
    return hipGetLastError();
}

// The rows of a workgroup, its waves side by side and the stages of X; is X there as a whole?
bool share(W4Args& a, int rows, int cus) {
    a.rows = rows;
    if (rows > 32) {
        a.wn = 8;
        a.kc = 512;
        return false;
    }
    // Waves side by side; the others share K.  As few as give no more workgroups than run at once: two on a compute
    // unit, or one where X takes more than half of its LDS (12 rows, 12288 x 4096: 384 workgroups of 96 KB take 14.5 us a
    // call in two rounds, 192 in one 10.5; the kernels alone under a trace 15.4 and 11.6).  A stage of X is a batch of each of the waves that share K, or all of K where it
    // fits.
    constexpr int waves = waves_of(1), batch = 128 * depth_of(1);
    for (a.wn = 1;; a.wn *= 2) {
        const int kc = batch * (waves / a.wn), all = a.K > 0 ? (a.K + kc - 1) / kc * kc : kc;
        const bool whole = (int64_t)rows * all * 2 <= 2 * kStageBytes;
        a.kc = whole ? all : kc;
        const bool fits = whole || rows * kc * 2 <= kStageBytes;
        const int at_once = rows * a.kc * 2 * (whole ? 1 : 2) <= 80 * 1024 ? 2 * cus : cus;
        if (a.wn == waves || (fits && (a.N + 16 * a.wn - 1) / (16 * a.wn) <= at_once)) return whole;
    }
}

template <class T, class TO, bool E2M1>
hipError_t by_rows(W4Args a, int cus, hipStream_t st) {
    // 64 rows to a workgroup, so that the weights pass once; fewer where that leaves more than half of the compute
    // units without one (the weights come out of a cache after the first time).  bf16, groups of 128, K = 4096: 48
    // rows, N = 4096 15.8 us, 25.5 with all rows in each of 32 workgroups; 32 rows, N = 12288 (192 workgroups)
    // 16.2, 23.4 with 16 rows to each of twice as many.
    int rows = a.M < 64 ? a.M : 64;
    bool whole = share(a, rows, cus);
    while (rows > 16 && (int64_t)((a.N + 16 * a.wn - 1) / (16 * a.wn)) * ((a.M + rows - 1) / rows) < cus / 2) {
        rows = rows > 32 ? 32 : 16;
        whole = share(a, rows, cus);
    }
    if (rows <= 16) return whole ? run<T, TO, E2M1, 1, false>(a, st) : run<T, TO, E2M1, 1, true>(a, st);
    if (rows <= 32) return whole ? run<T, TO, E2M1, 2, false>(a, st) : run<T, TO, E2M1, 2, true>(a, st);
    return rows <= 48 ? run<T, TO, E2M1, 3, true>(a, st) : run<T, TO, E2M1, 4, true>(a, st);
}

template <class T>
hipError_t by_type(const W4Args& a, bool e2m1, bool out_f32, int cus, hipStream_t st) {
    if (e2m1) return out_f32 ? by_rows<T, float, true>(a, cus, st) : by_rows<T, T, true>(a, cus, st);
    return out_f32 ? by_rows<T, float, false>(a, cus, st) : by_rows<T, T, false>(a, cus, st);
}

static_assert(128 * depth_of(4) * waves_of(4) / 8 == 512 && 64 * 512 * 2 <= kStageBytes &&
                  32 * 128 * depth_of(2) * 2 <= kStageBytes,
              "a stage of all rows, for waves side by side");

}  // namespace

hipError_t launch_gemm_w4(const W4Args& a, int32_t dtype, bool e2m1, bool out_f32, int cus, hipStream_t st) {
    return dtype == 1 ? by_type<__bf16>(a, e2m1, out_f32, cus, st) : by_type<_Float16>(a, e2m1, out_f32, cus, st);
}

}  // namespace tcm
