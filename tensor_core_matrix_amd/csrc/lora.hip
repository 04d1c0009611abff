// One projection with the low-rank adapters of many requests beside it:
// Out[i] = X[i] W^T + s_a (X[i] A_a^T) B_a^T, a the adapter of row i.
//
// Two launches.  lora_shrink_kernel computes t = s_a (X A_a^T) for the rows that
// have an adapter; the product kernel adds t B_a^T to its accumulators before
// the one rounding (lora_tail.h).
#include <type_traits>

#include "layer_internal.h"
#include "lora_tail.h"
#include "tcm_device.h"

namespace tcm {

namespace {

// ---- t = s_a (X A_a^T) ----------------------------------------------------------
// A workgroup takes a block of 16 rows, and of the adapters that they name those
// whose first row in the block is blockIdx.x % slots (+ slots, ...).  Per adapter
// the 16 rows are multiplied by A_a on the matrix cores, eight waves taking
// 32-deep steps in turn, and the rows that name it keep the result.  Bound by
// reading A (each adapter once per block that names it).
template <class T, int RB>
__global__ __launch_bounds__(512) void lora_shrink_kernel(LoraArgs p, int slots) {
    typedef LoraMma<T> O;
    typedef typename O::x8 x8;
    __shared__ __attribute__((aligned(16))) float red[8][16][RB * 16 + 4];
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (int)(blockIdx.x / slots) * 16, s0 = blockIdx.x % slots;
    const int k0 = blockIdx.y * p.kpart, k1 = min(p.K, k0 + p.kpart);
    const int id = lora_row(p, m0, r16);
    uint32_t left = (uint32_t)__ballot(id >= 0) & 0xffffu;
    const T* xr = (const T*)p.X + (int64_t)min(m0 + r16, p.M - 1) * p.ldx + 8 * g4;
    while (left) {
        const int first = __builtin_ctz(left);
        const int a = __builtin_amdgcn_readlane(id, first);
        const uint32_t rows = (uint32_t)__ballot(id == a) & 0xffffu;
        left &= ~rows;
        if (first % slots != s0) continue;
        const int rank = lora_rank(p, a);
        f32x4_t acc[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[i] = (f32x4_t){};
        const T* ar[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i)
            ar[i] = (const T*)p.A + ((int64_t)a * p.R + min(16 * i + r16, p.R - 1)) * p.K + 8 * g4;
        constexpr int U = RB <= 2 ? 4 : 2;
        int k = k0 + 32 * wave;
        for (; k + 256 * (U - 1) + 32 <= k1; k += 256 * U) {
            x8 x[U], f[U][RB];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                x[u] = *(const x8*)(xr + k + 256 * u);
#pragma unroll
                for (int i = 0; i < RB; ++i) f[u][i] = *(const x8*)(ar[i] + k + 256 * u);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < RB; ++i) acc[i] = O::mma(f[u][i], x[u], acc[i]);
        }
        for (; k < k1; k += 256) {  // (the last step may be cut by K)
            const bool in = k + 8 * g4 < k1;
            const x8 x = in ? *(const x8*)(xr + k) : (x8){};
#pragma unroll
            for (int i = 0; i < RB; ++i)
                acc[i] = O::mma(in ? *(const x8*)(ar[i] + k) : (x8){}, x, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) *(f32x4_t*)&red[wave][r16][16 * i + 4 * g4] = acc[i];
        __syncthreads();
        const float scale = p.scales ? p.scales[a] : 1.0f;
        for (int x = threadIdx.x; x < 16 * RB * 16; x += 512) {
            const int row = x / (RB * 16), r = x % (RB * 16);
            if (!((rows >> row) & 1u) || r >= p.R) continue;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) s += red[w][row][r];
            p.t[((int64_t)blockIdx.y * p.M + m0 + row) * p.R + r] = r < rank ? s * scale : 0.0f;
        }
        __syncthreads();
    }
}

// ---- few rows ---------------------------------------------------------------------
// Bound by reading W once.  A workgroup owns 16 NB output columns for all 16 MB >= M
// rows; its eight waves take the 32-deep K steps in turn, reading W from memory
// straight into operand registers (no element of W is used twice), and their
// sums meet in LDS.  The adapters are dealt to the waves too: what an adapter adds
// to a block of rows is one more term of that sum.
template <class T, class TO, int MB, int NB>
__global__ __launch_bounds__(512) void lora_rows_kernel(LoraArgs p) {
    typedef LoraMma<T> O;
    typedef typename O::x8 x8;
    __shared__ __attribute__((aligned(16))) f32x4_t red[8][MB * NB][64];
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * NB;
    f32x4_t acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = (f32x4_t){};
    const T* wr[NB];
    const T* xr[MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
        wr[j] = (const T*)p.W + (int64_t)min(n0 + 16 * j + r16, p.N - 1) * p.K + 8 * g4;
#pragma unroll
    for (int i = 0; i < MB; ++i)
        xr[i] = (const T*)p.X + (int64_t)min(16 * i + r16, p.M - 1) * p.ldx + 8 * g4;
    constexpr int U = 8 / NB;
    int k = 32 * wave;
    for (; k + 256 * (U - 1) + 32 <= p.K; k += 256 * U) {
        x8 w[U][NB];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NB; ++j) w[u][j] = *(const x8*)(wr[j] + k + 256 * u);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                const x8 x = *(const x8*)(xr[i] + k + 256 * u);
#pragma unroll
                for (int j = 0; j < NB; ++j) acc[i][j] = O::mma(w[u][j], x, acc[i][j]);
            }
    }
    for (; k < p.K; k += 256) {
        const bool in = k + 8 * g4 < p.K;
        x8 w[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) w[j] = in ? *(const x8*)(wr[j] + k) : (x8){};
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const x8 x = in ? *(const x8*)(xr[i] + k) : (x8){};
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = O::mma(w[j], x, acc[i][j]);
        }
    }
    int turn = 0;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int id = lora_row(p, 16 * i, r16);
        uint32_t left = (uint32_t)__ballot(id >= 0) & 0xffffu;
        while (left) {
            const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
            left &= ~(uint32_t)__ballot(id == a);
            if ((turn++ & 7) != wave) continue;
            const int rank = lora_rank(p, a);
            f32x4_t d[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) d[j] = (f32x4_t){};
            for (int r0 = 0; r0 < rank; r0 += 16) {
                const x8 t = lora_t<T>(p, 16 * i + r16, r0, g4, id == a);
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    d[j] = O::mma(lora_b<T>(p, a, rank, n0 + 16 * j + r16, r0, g4), t, d[j]);
            }
            if (id == a)
#pragma unroll
                for (int j = 0; j < NB; ++j) acc[i][j] += d[j];
        }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) red[wave][i * NB + j][lane] = acc[i][j];
    __syncthreads();
    for (int x = threadIdx.x; x < MB * NB * 64; x += 512) {
        const int blk = x >> 6, l = x & 63;
        f32x4_t s = red[0][blk][l];
#pragma unroll
        for (int w = 1; w < 8; ++w) s += red[w][blk][l];
        const int m = 16 * (blk / NB) + (l & 15), n = n0 + 16 * (blk % NB) + 4 * (l >> 4);
        if (m >= p.M) continue;
        TO* row = (TO*)p.out + (int64_t)m * p.ldo;
        if (n + 3 < p.N && (p.ldo & 3) == 0) {
            store4<TO>(row + n, s[0], s[1], s[2], s[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N) row[n + e] = convert_out<TO>(s[e]);
        }
    }
}

// ---- many rows ----------------------------------------------------------------------
// BM x BN tiles, four waves in a 2 x 2 arrangement, 64-deep slices by DMA into a ring
// of S stages (128-byte rows whose 16-byte chunk c lies at c ^ (row / 2) % 8, so that
// 16 rows' reads meet 16 bank groups), one barrier a slice.
template <class T, class TO, int BM, int BN, int S>
__global__ __launch_bounds__(256) void lora_tile_kernel(LoraArgs p, int tiles_m, int tiles_n) {
    typedef LoraMma<T> O;
    typedef typename O::x8 x8;
    constexpr int STAGE = (BM + BN) * 128, CA = BM / 32, CB = BN / 32, C = CA + CB;
    constexpr int FM = BM / 32, FN = BN / 32;
    __shared__ __attribute__((aligned(1024))) char lds[S * STAGE];
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    // tiles down groups of 4 tile rows, neighbours on one XCD
    GemmArgs order;
    order.tiles_m = tiles_m;
    order.tiles_n = tiles_n;
    order.tiles_per_batch = tiles_m * tiles_n;
    order.group_m = 4;
    int batch, tm, tn;
    tile_coords(order, logical_block(blockIdx.x, gridDim.x), batch, tm, tn);
    const int rows_a = min(BM, p.M - tm * BM), rows_b = min(BN, p.N - tn * BN);
    const uint32_t lda = (uint32_t)p.ldx * 2u, ldb = (uint32_t)p.K * 2u;
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc((const char*)p.X + (int64_t)tm * BM * lda, (uint32_t)(rows_a - 1) * lda + ldb);
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc((const char*)p.W + (int64_t)tn * BN * ldb, (uint32_t)rows_b * ldb);
    const int cp_row = wave * 8 + lane / 8;
    const int cp_chunk = (lane & 7) ^ ((cp_row >> 1) & 7);
    const int ksteps = (p.K + 63) / 64;
    auto issue = [&](int g) {
        const bool in = g < ksteps && g * 64 + cp_chunk * 8 < p.K;
        const uint32_t at = (uint32_t)g * 128u + (uint32_t)cp_chunk * 16u;
        char* dst = lds + (g % S) * STAGE + wave * 1024;
#pragma unroll
        for (int x = 0; x < CA; ++x)
            // (rows past the tile's last are past the buffer's end, or hold K
            // values of the next row that no output uses)
            copy16_to_lds(ra, dst + x * 4096,
                          in && 32 * x + cp_row < rows_a ? (uint32_t)(32 * x + cp_row) * lda + at : kOutOfRange);
#pragma unroll
        for (int x = 0; x < CB; ++x)
            copy16_to_lds(rb, dst + (CA + x) * 4096,
                          in ? (uint32_t)(32 * x + cp_row) * ldb + at : kOutOfRange);
    };
    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4_t){};
#pragma unroll
    for (int g = 0; g < S - 1; ++g) issue(g);
    const int xr = r16 >> 1;
    for (int g = 0; g < ksteps; ++g) {
        wait_vmcnt<(S - 2) * C>();
        barrier_lds();
        issue(g + S - 1);
        const char* st = lds + (g % S) * STAGE;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int ch = ((4 * s + g4) ^ xr) * 16;
            x8 fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                fa[i] = *(const x8*)(st + (wm * (BM / 2) + 16 * i + r16) * 128 + ch);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fb[j] = *(const x8*)(st + (BM + wn * (BN / 2) + 16 * j + r16) * 128 + ch);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = O::mma(fb[j], fa[i], acc[i][j]);
        }
    }
    wait_vmcnt<0>();  // (copies of slices past the last: zeros, but still on their way)
    const int m0 = tm * BM + wm * (BM / 2), n0 = tn * BN + wn * (BN / 2);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int id = lora_row(p, m0 + 16 * i, r16);
        uint32_t left = (uint32_t)__ballot(id >= 0) & 0xffffu;
        while (left) {
            const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
            left &= ~(uint32_t)__ballot(id == a);
            const int rank = lora_rank(p, a);
            f32x4_t d[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) d[j] = (f32x4_t){};
            for (int r0 = 0; r0 < rank; r0 += 16) {
                const x8 t = lora_t<T>(p, m0 + 16 * i + r16, r0, g4, id == a);
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    d[j] = O::mma(lora_b<T>(p, a, rank, n0 + 16 * j + r16, r0, g4), t, d[j]);
            }
            if (id == a)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] += d[j];
        }
    }
    const bool vec = (p.ldo & 3) == 0;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + 16 * i + r16;
        if (m >= p.M) continue;
        TO* row = (TO*)p.out + (int64_t)m * p.ldo;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int n = n0 + 16 * j + 4 * g4;
            const f32x4_t v = acc[i][j];
            if (vec && n + 3 < p.N) {
                store4<TO>(row + n, v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N) row[n + e] = convert_out<TO>(v[e]);
            }
        }
    }
}

int cdiv_i(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <class T, int RB>
void shrink(const LoraArgs& a, hipStream_t st) {
    // few rows: an adapter a workgroup; many: a block's adapters in turn
    const int slots = a.M <= 256 ? 16 : 1;
    hipLaunchKernelGGL((lora_shrink_kernel<T, RB>), dim3(cdiv_i(a.M, 16) * slots, a.ksplit), dim3(512), 0,
                       st, a, slots);
}

template <class T, class TO, int BM, int BN, int S>
void tiles(const LoraArgs& a, hipStream_t st) {
    const int tm = cdiv_i(a.M, BM), tn = cdiv_i(a.N, BN);
    hipLaunchKernelGGL((lora_tile_kernel<T, TO, BM, BN, S>), dim3(tm * tn), dim3(256), 0, st, a, tm, tn);
}

template <class T, class TO>
void product(const LoraArgs& a, int cus, hipStream_t st) {
    if (a.M <= 16)
        hipLaunchKernelGGL((lora_rows_kernel<T, TO, 1, 1>), dim3(cdiv_i(a.N, 16)), dim3(512), 0, st, a);
    else if (a.M <= 32)
        hipLaunchKernelGGL((lora_rows_kernel<T, TO, 2, 1>), dim3(cdiv_i(a.N, 16)), dim3(512), 0, st, a);
    else if (a.M <= 64)
        hipLaunchKernelGGL((lora_rows_kernel<T, TO, 4, 2>), dim3(cdiv_i(a.N, 32)), dim3(512), 0, st, a);
    else if ((int64_t)cdiv_i(a.M, 128) * cdiv_i(a.N, 128) >= cus)
        tiles<T, TO, 128, 128, 2>(a, st);
    else
        tiles<T, TO, 64, 64, 4>(a, st);
}

template <class T>
hipError_t run(const LoraArgs& a, int32_t out_dtype, int cus, hipStream_t st) {
    if (a.L > 0 && a.R > 0 && a.K > 0) {
        if (a.R <= 16) shrink<T, 1>(a, st);
        else if (a.R <= 32) shrink<T, 2>(a, st);
        else if (a.R <= 64) shrink<T, 4>(a, st);
        else shrink<T, 8>(a, st);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (out_dtype == 2) product<T, float>(a, cus, st);
    else product<T, T>(a, cus, st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraArgs& a, int32_t dtype, int32_t out_dtype, int cus, hipStream_t st) {
    return dtype == 1 ? run<__bf16>(a, out_dtype, cus, st) : run<_Float16>(a, out_dtype, cus, st);
}

}  // namespace tcm
