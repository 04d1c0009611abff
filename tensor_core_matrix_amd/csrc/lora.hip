// One projection with the low-rank adapters of many requests beside it:
// Out[i] = X[i] W^T + s_a (X[i] A_a^T) B_a^T, a the adapter of row i.
//
// Two launches.  lora_shrink_kernel computes t = s_a (X A_a^T) for the rows that
// have an adapter; the product kernel adds t B_a^T to its accumulators before
// the one rounding (lora_tail.h).  Up to 64 rows the product is bound by reading W
// (lora_rows_kernel: one row of 4096 x 4096 3.3 + 8.5 us, 3.9 TB/s; 48 rows of 8192 x
// 4096 with nearly as many adapters of rank 32 6.2 + 31 us, 23 without adapters), beyond
// them by what a compute unit reads into LDS and then by the matrix cores
// (lora_tile_kernel: 333 rows of 4096 x 4096 5.3 + 29 us, 25 without adapters; 4096 rows
// 12 + 125 us as traced and 128 a call among others, 120 without adapters).
#include <type_traits>

#include "layer_internal.h"
#include "lora_tail.h"
#include "tcm_device.h"

namespace tcm {

namespace {

// 16 rows x 256 bytes in LDS, row after row; 16 bytes c of a row lie at c ^ row, so
// that 16 rows' reads of one piece meet 16 groups of banks.
__device__ __forceinline__ void* piece_at(char* area, int row, int c) {
    return area + row * 256 + ((c ^ row) * 16);
}

// ---- t = s_a (X A_a^T) ----------------------------------------------------------
// A workgroup takes a block of 16 rows and a part of K, and of the adapters that the
// rows name those whose first row in the block is blockIdx.x % slots (+ slots, ...).
// Per adapter the 16 rows are multiplied by A_a on the matrix cores, eight waves
// taking 128-deep pieces of K in turn, and the rows that name it keep the result.
// Bound by reading X and A, which come in whole 256-byte stretches of their rows and
// are turned into operands through a wave's own LDS areas: rows are often a power
// of two apart, and the operand's own 16 rows x 64 bytes then meet few channels
// (4096 rows of 8 KiB: 12 us, and 20 that way).
template <class T, int RB>
__global__ __launch_bounds__(512) void lora_shrink_kernel(LoraArgs p, int slots) {
    typedef LoraMma<T> O;
    typedef typename O::x8 x8;
    constexpr int RED = 8 * 16 * (RB * 16 + 4) * 4, AREAS = 8 * 2 * 4096;
    __shared__ __attribute__((aligned(1024))) char lds[RED > AREAS ? RED : AREAS];
    float(*const red)[16][RB * 16 + 4] = (float(*)[16][RB * 16 + 4])lds;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (int)(blockIdx.x / slots) * 16, s0 = blockIdx.x % slots;
    const int k0 = blockIdx.y * p.kpart, k1 = min(p.K, k0 + p.kpart);
    const int id = lora_row(p, m0, r16);
    uint32_t left = (uint32_t)__ballot(id >= 0) & 0xffffu;
    char* const xa = lds + wave * 8192;
    char* const aa = xa + 4096;
    // lane: row 4 x + lane / 16 of 16, 16 bytes lane % 16
    auto load = [&](i32x4_t (&v)[4], const T* base, int rows, int64_t ld, int k) {
        const bool in = k + 8 * r16 < k1;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            v[x] = in ? *(const i32x4_t*)(base + min(4 * x + g4, rows - 1) * ld + k + 8 * r16) : (i32x4_t){};
    };
    auto store = [&](char* area, const i32x4_t (&v)[4]) {
#pragma unroll
        for (int x = 0; x < 4; ++x) *(i32x4_t*)piece_at(area, 4 * x + g4, r16) = v[x];
    };
    while (left) {
        const int first = __builtin_ctz(left);
        const int a = __builtin_amdgcn_readlane(id, first);
        const uint32_t rows = (uint32_t)__ballot(id == a) & 0xffffu;
        left &= ~rows;
        if (first % slots != s0) continue;
        const int rank = lora_rank(p, a);
        const T* const xb = (const T*)p.X + (int64_t)m0 * p.ldx;
        const T* const ab = (const T*)p.A + (int64_t)a * p.R * p.K;
        f32x4_t acc[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[i] = (f32x4_t){};
        constexpr int AN = RB < 2 ? RB : 2;  // blocks of 16 ranks read at once
        for (int k = k0 + 128 * wave; k < k1; k += 1024) {
            i32x4_t xv[4];
            load(xv, xb, min(16, p.M - m0), p.ldx, k);
#pragma unroll
            for (int i0 = 0; i0 < RB; i0 += AN) {
                i32x4_t av[AN][4];
#pragma unroll
                for (int i = 0; i < AN; ++i)
                    if (16 * (i0 + i) < p.R)
                        load(av[i], ab + (int64_t)16 * (i0 + i) * p.K, min(16, p.R - 16 * (i0 + i)), p.K, k);
                wave_lds_exchange();
                if (i0 == 0) store(xa, xv);
#pragma unroll
                for (int i = 0; i < AN; ++i) {
                    if (16 * (i0 + i) >= p.R) continue;
                    store(aa, av[i]);
                    wave_lds_exchange();
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        acc[i0 + i] = O::mma(*(const x8*)piece_at(aa, r16, 4 * s + g4),
                                             *(const x8*)piece_at(xa, r16, 4 * s + g4), acc[i0 + i]);
                    wave_lds_exchange();
                }
            }
        }
        __syncthreads();  // (the areas end here)
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

constexpr int kNonTemporal = 2;  // cache policy of a buffer load: read once

// ---- few rows ---------------------------------------------------------------------
// Bound by reading W once.  A workgroup owns 16 NB output columns for all 16 MB >= M
// rows.  WW of its sixteen waves take W, pieces of K in turn: whole stretches of its
// rows (a probe reads 6.4 TB/s that way, and 5.2 in the operand's own pattern of 16
// rows x 64 bytes), which a wave turns into operands through its own LDS area, the
// next piece on its way while one is multiplied.  The other waves take what the
// adapters add, a row a wave in turn: with few rows nearly every row has an
// adapter of its own, so there is nothing for the matrix cores to share, and a
// row's 16 NB dot products over the ranks are done by its lanes, in fp32 and from
// nothing but the row's own adapter.  Everything meets in LDS at the end.
template <class T, class TO, int MB, int NB>
__global__ __launch_bounds__(1024) void lora_rows_kernel(LoraArgs p) {
    typedef LoraMma<T> O;
    typedef typename O::x8 x8;
    constexpr int WW = 8, LW = 16 - WW;        // waves that take W, and adapters
    constexpr int PB = 256 / NB;               // bytes of a row's piece,
    constexpr int PK = PB / 2, S = PK / 32;    // its K values and 32-deep steps
    constexpr int LR = PB / 16, RN = 64 / LR;  // lanes that read it, rows of one read
    constexpr int AREA = 4096;
    __shared__ __attribute__((aligned(1024))) char areas[WW * AREA];
    __shared__ __attribute__((aligned(1024))) f32x4_t red[WW + 1][MB * NB][64];
    __shared__ __attribute__((aligned(16))) float ts[LW][4][kLoraMaxRank];
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * NB;
    if (wave < WW) {
        f32x4_t acc[MB][NB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = (f32x4_t){};
        // lane: row RN x + lane / LR of the columns' rows, 16 bytes lane % LR; past the
        // last row or K the buffers give zeros
        const int wc = lane % LR, wr = lane / LR;
        const uint32_t wrow = (uint32_t)p.K * 2u, xrow = (uint32_t)p.ldx * 2u;
        const __amdgpu_buffer_rsrc_t rw = make_rsrc((const T*)p.W + (int64_t)n0 * p.K,
                                                    (uint32_t)min(16 * NB, p.N - n0) * wrow);
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.X, (uint32_t)(p.M - 1) * xrow + wrow);
        const uint32_t w0 = (uint32_t)wr * wrow + 16u * wc, x0 = (uint32_t)r16 * xrow + 16u * g4;
        char* const area = areas + wave * AREA;
        // 16 bytes c of a row lie at c ^ swz(row): 16 rows' reads meet 16 bank groups
        auto swz = [](int row) { return LR == 16 ? row & 15 : (row >> 1) & 7; };
        auto load = [&](i32x4_t (&w)[4], int k) {
            const uint32_t at = k + 8 * wc < p.K ? w0 + 2u * (uint32_t)k : kOutOfRange;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                w[x] = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                       rw, at + (uint32_t)(RN * x) * wrow, 0, kNonTemporal));
        };
        // X comes from the caches, its reads ahead of the next piece's of W: a wave's
        // loads return in order, and W's would be waited for with them
        x8 xf[S][MB];
        auto load_x = [&](int k) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint32_t at = k + 32 * s + 8 * g4 < p.K ? x0 + 2u * (uint32_t)(k + 32 * s) : kOutOfRange;
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    // (a row past M may lie before the buffer's end)
                    const uint32_t row = 16 * i + r16 < p.M ? at + (uint32_t)(16 * i) * xrow : kOutOfRange;
                    xf[s][i] = __builtin_bit_cast(x8, __builtin_amdgcn_raw_buffer_load_b128(rx, row, 0, 0));
                }
            }
        };
        auto multiply = [&](const i32x4_t (&w)[4]) {
            wave_lds_exchange();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int row = RN * x + wr;
                *(i32x4_t*)(area + row * PB + ((wc ^ swz(row)) * 16)) = w[x];
            }
            wave_lds_exchange();
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const x8 f = *(const x8*)(area + (16 * j + r16) * PB + (((4 * s + g4) ^ swz(r16)) * 16));
#pragma unroll
                    for (int i = 0; i < MB; ++i) acc[i][j] = O::mma(f, xf[s][i], acc[i][j]);
                }
        };
        i32x4_t wa[4], wb[4];
        int k = PK * wave;
        constexpr int STEP = PK * WW;
        if (k < p.K) load(wa, k);
        while (k < p.K) {
            load_x(k);
            if (k + STEP < p.K) load(wb, k + STEP);
            multiply(wa);
            k += STEP;
            if (k >= p.K) break;
            load_x(k);
            if (k + STEP < p.K) load(wa, k + STEP);
            multiply(wb);
            k += STEP;
        }
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) red[wave][i * NB + j][lane] = acc[i][j];
    } else {
        // lane: column lane % C and the ranks 8 (lane / C), + 8 P, .. of it
        constexpr int C = 16 * NB, P = 64 / C;
        const int lw = wave - WW, c = lane % C, part = lane / C;
        const int n = min(n0 + c, p.N - 1);
        // row m's sum for column c in the layout of the products' sums
        auto put = [&](int m, float v) {
            float* at = (float*)&red[WW][(m >> 4) * NB + (c >> 4)][(m & 15) + 16 * ((c & 15) >> 2)];
            if (part == 0) at[c & 3] = v;
        };
        const int id = lora_row(p, 0, lane);  // of row `lane`
        // four rows at a time, all their reads under way together: the first BN
        // pieces of B_a's row, and t (the parts of K summed, lane r rank r), which
        // goes through LDS (the wave's own: its operations run in order)
        constexpr int BN = 2, QN = 4;
        for (int m0 = lw; m0 < 16 * MB; m0 += QN * LW) {
            int a[QN], rank[QN];
            x8 b[QN][BN];
            float t[QN][kLoraMaxRank / 64];
            const T* br[QN];
#pragma unroll
            for (int q = 0; q < QN; ++q) {
                const int m = m0 + q * LW;
                a[q] = m < 16 * MB ? __builtin_amdgcn_readlane(id, m & 63) : -1;
                rank[q] = a[q] >= 0 ? lora_rank(p, a[q]) : 0;
            }
#pragma unroll
            for (int q = 0; q < QN; ++q) {
                br[q] = (const T*)p.B + ((int64_t)max(a[q], 0) * p.N + n) * p.R + 8 * part;
#pragma unroll
                for (int i = 0; i < BN; ++i)
                    b[q][i] = 8 * (part + P * i) < rank[q] ? *(const x8*)(br[q] + 8 * P * i) : (x8){};
            }
#pragma unroll
            for (int q = 0; q < QN; ++q)
#pragma unroll
                for (int h = 0; h < kLoraMaxRank / 64; ++h) {
                    const int r = lane + 64 * h;
                    float v = 0.0f;
                    if (r < rank[q]) {
                        const float* tr = p.t + (int64_t)(m0 + q * LW) * p.R + r;
                        for (int s = 0; s < p.ksplit; s += 4) {
                            float u[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                u[x] = tr[(int64_t)min(s + x, p.ksplit - 1) * p.M * p.R];
#pragma unroll
                            for (int x = 0; x < 4; ++x) v += s + x < p.ksplit ? u[x] : 0.0f;
                        }
                    }
                    t[q][h] = v;
                }
            wave_lds_exchange();
#pragma unroll
            for (int q = 0; q < QN; ++q)
#pragma unroll
                for (int h = 0; h < kLoraMaxRank / 64; ++h) ts[lw][q][lane + 64 * h] = t[q][h];
            wave_lds_exchange();
#pragma unroll
            for (int q = 0; q < QN; ++q) {
                float sum = 0.0f;
                for (int i0 = 0; 8 * P * i0 < rank[q]; i0 += BN) {
                    if (i0 > 0)
#pragma unroll
                        for (int i = 0; i < BN; ++i)
                            b[q][i] = 8 * (part + P * (i0 + i)) < rank[q] ? *(const x8*)(br[q] + 8 * P * (i0 + i))
                                                                          : (x8){};
#pragma unroll
                    for (int i = 0; i < BN; ++i) {
                        const int r = 8 * (part + P * (i0 + i));
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            sum += r + e < rank[q] ? ts[lw][q][r + e] * (float)b[q][i][e] : 0.0f;
                    }
                }
#pragma unroll
                for (int x = C; x < 64; x *= 2) sum += __shfl_xor(sum, x);
                if (m0 + q * LW < 16 * MB) put(m0 + q * LW, sum);
            }
            wave_lds_exchange();
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < MB * NB * 64; x += 1024) {
        const int blk = x >> 6, l = x & 63;
        f32x4_t s = red[0][blk][l];
#pragma unroll
        for (int w = 1; w < WW + 1; ++w) s += red[w][blk][l];
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
// BM x BN tiles, WM x WN waves, 64-deep slices by DMA into a ring of S stages (128-byte
// rows whose 16-byte chunk c lies at c ^ (row / 2) % 8, so that 16 rows' reads meet 16
// bank groups), one barrier a slice.  Where tiles are small, KG such groups of waves,
// each with a ring, take every KG-th slice side by side and their sums meet in LDS,
// so that one group's products and reads cover another's wait and barrier (without
// adapters, 128 rows of 4096 x 4096 in 64 x 64 tiles: 21 us with one group, 17 with two;
// 333 rows in 128 x 64 tiles: 26 and 25).  A compute unit then reads about 65 GB/s into
// LDS, in tiles of any size, rings of any depth: that is the bound of these.
template <class T, class TO, int BM, int BN, int S, int WM, int WN, int KG>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void lora_tile_kernel(LoraArgs p, int tiles_m, int tiles_n) {
    typedef LoraMma<T> O;
    typedef typename O::x8 x8;
    constexpr int WV = WM * WN, ROWS = 8 * WV;  // rows of one copy by all waves
    constexpr int STAGE = (BM + BN) * 128, CA = BM / ROWS, CB = BN / ROWS, C = CA + CB;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    static_assert((ROWS / 2) % 8 == 0 || ROWS % 16 == 0, "a lane's chunk is the same in every copy");
    __shared__ __attribute__((aligned(1024))) char all[KG * S * STAGE];
    static_assert(KG == 1 || (KG - 1) * BM * BN * 4 <= KG * S * STAGE, "the groups' sums meet in the rings");
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = wave_all / WV, wave = wave_all % WV;
    char* const lds = all + kg * S * STAGE;
    const int wm = wave / WN, wn = wave % WN;
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
    const int ksteps = (p.K + 64 * KG - 1) / (64 * KG);  // slices of each group
    auto issue = [&](int g) {
        const int slice = g * KG + kg;
        const bool in = g < ksteps && slice * 64 + cp_chunk * 8 < p.K;
        const uint32_t at = (uint32_t)slice * 128u + (uint32_t)cp_chunk * 16u;
        char* dst = lds + (g % S) * STAGE + wave * 1024;
#pragma unroll
        for (int x = 0; x < CA; ++x)
            // (rows past the tile's last are past the buffer's end, or hold K
            // values of the next row that no output uses)
            copy16_to_lds(ra, dst + x * ROWS * 128,
                          in && ROWS * x + cp_row < rows_a ? (uint32_t)(ROWS * x + cp_row) * lda + at
                                                           : kOutOfRange);
#pragma unroll
        for (int x = 0; x < CB; ++x)
            copy16_to_lds(rb, dst + (CA + x) * ROWS * 128,
                          in ? (uint32_t)(ROWS * x + cp_row) * ldb + at : kOutOfRange);
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
                fa[i] = *(const x8*)(st + (wm * (BM / WM) + 16 * i + r16) * 128 + ch);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fb[j] = *(const x8*)(st + (BM + wn * (BN / WN) + 16 * j + r16) * 128 + ch);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = O::mma(fb[j], fa[i], acc[i][j]);
        }
    }
    wait_vmcnt<0>();  // (copies of slices past the last: zeros, but still on their way)
    const int m0 = tm * BM + wm * (BM / WM), n0 = tn * BN + wn * (BN / WN);
    constexpr bool FULL = sizeof(TO) == 4 && std::is_same<T, __bf16>::value;
    if (KG == 1 || kg == KG - 1) {
        if constexpr (FM * FN >= 32)
            lora_add_lean<T, FULL>(p, acc, m0, n0);
        else
            lora_add<T, FULL>(p, acc, m0, n0);
    }
    if constexpr (KG > 1) {
        __syncthreads();  // (the rings end here)
        f32x4_t(*const sum)[FM * FN][64] = (f32x4_t(*)[FM * FN][64])all;
        if (kg > 0)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) sum[(kg - 1) * WV + wave][i * FN + j][lane] = acc[i][j];
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int x = 0; x < KG - 1; ++x)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] += sum[x * WV + wave][i * FN + j][lane];
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

template <class T, class TO, int BM, int BN, int S, int WM, int WN, int KG>
void tiles(const LoraArgs& a, hipStream_t st) {
    const int tm = cdiv_i(a.M, BM), tn = cdiv_i(a.N, BN);
    hipLaunchKernelGGL((lora_tile_kernel<T, TO, BM, BN, S, WM, WN, KG>), dim3(tm * tn), dim3(64 * WM * WN * KG), 0,
                       st, a, tm, tn);
}

template <class T, class TO, int MB, int NB>
void rows(const LoraArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((lora_rows_kernel<T, TO, MB, NB>), dim3(cdiv_i(a.N, 16 * NB)), dim3(1024), 0, st, a);
}

template <class T, class TO>
void product(const LoraArgs& a, int cus, hipStream_t st) {
    // Few rows.  32 columns a workgroup read X half as often as 16, which counts from
    // two blocks of rows on, where they still give every compute unit a workgroup
    // (N = 8192: 48 rows 37 us, and 51 with 16; one row 21, and 16 with 16;
    // N = 4096, 48 rows: 33, and 30 with 16).
    const int mb = cdiv_i(a.M, 16);
    const bool wide = mb > 1 && cdiv_i(a.N, 32) >= cus;
    if (mb <= 4) {
        switch (2 * mb + wide) {
        case 2: rows<T, TO, 1, 1>(a, st); break;
        case 4: rows<T, TO, 2, 1>(a, st); break;
        case 5: rows<T, TO, 2, 2>(a, st); break;
        case 6: rows<T, TO, 3, 1>(a, st); break;
        case 7: rows<T, TO, 3, 2>(a, st); break;
        case 8: rows<T, TO, 4, 1>(a, st); break;
        case 9: rows<T, TO, 4, 2>(a, st); break;
        }
    }
    if (mb <= 4) return;
    // The largest tile that still gives every compute unit one (128 x 64: three in
    // four of them), as what a unit reads into LDS is what bounds the small ones; and
    // of 256 x 256, which are one a unit at a time, not so few in the last round that
    // more than a quarter of the rounds idles.  us with an adapter a request, rank 16,
    // K = 4096:
    //   256 x 256 and 128 x 128: 4096 x 4096 (256 tiles) 129 and 156; 4352 x 4096 (272) 224
    //     and 176; 6144 x 4096 (384) 229 and 222; 6400 x 4096 (400) 231 and 245; 8192 x 4096
    //     (512) 249 and 298; 8448 x 4096 (528) 344 and 315; 9984 x 4096 (624) 345 and 357
    //   128 x 128 and 128 x 64: 2048 x 2048 (256 tiles) 55 and 58; 4096 x 2048 81 and 110
    //   128 x 64 and 64 x 64: 333 x 4096 (192 tiles) 33 and 40; 256 x 4096 (128) 33 and 25
    auto count = [&](int64_t bm, int64_t bn) { return (int64_t)cdiv_i(a.M, bm) * cdiv_i(a.N, bn); };
    const int64_t large = count(256, 256), rounds = cdiv_i(large, cus);
    if (large >= cus && 4 * large > 3 * rounds * cus)
        tiles<T, TO, 256, 256, 2, 4, 2, 1>(a, st);
    else if (count(128, 128) >= cus)
        tiles<T, TO, 128, 128, 2, 2, 2, 1>(a, st);
    else if (4 * count(128, 64) >= 3 * cus)
        tiles<T, TO, 128, 64, 3, 4, 2, 2>(a, st);
    else
        tiles<T, TO, 64, 64, 4, 4, 2, 2>(a, st);
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
