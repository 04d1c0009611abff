/*
 * tcm.h -- C ABI of libtcm, a tiled dense matrix product Out = A . B^T for
 * AMD Instinct MI355X (gfx950), written in HIP for the CDNA4 matrix cores.
 *
 * The operation is the one the pages state:
 *   - "Blackwell Tensor Cores" (TVM TIRx guide), "The Accumulator's Lifetime":
 *     Out = A @ B.T, float16 inputs, float32 accumulation and output; the
 *     first MMA of a tile ignores the accumulator, so Out is overwritten
 *     (there is no C input and no alpha/beta).
 *   - "API Card: Blackwell Pipeline (tcgen05)" (cuBLASDx), "Descriptor." and
 *     "Host side.": row-major A (M x K), column-major B (K x N, i.e. stored
 *     N x K, "K-major"), row-major C (the TN arrangement); 16-byte alignment
 *     of A, B and C; bfloat16 inputs with float accumulation; batched
 *     problems as in its batched example.
 *   - "Hopper and Blackwell GEMM", Concept "FP8 and FP4, with block scaling"
 *     and its format table: MXFP8 = E4M3 elements with one E8M0 (power of
 *     two) scale per 32 consecutive elements of every row of A and column of
 *     B^T, the scales applied inside the product.
 *
 * Conventions shared by every entry point
 *   Layout     A: M x K row-major (leading dimension K).  B: N x K row-major
 *              (leading dimension K).  Out: M x N row-major (leading dimension
 *              N).  Batched operands are contiguous: problem p starts at
 *              p*M*K, p*N*K and p*M*N elements.  tcm_gemm alone takes other
 *              arrangements and leading dimensions.
 *   Pointers   device pointers (hipMalloc'ed or torch CUDA tensors) on the
 *              current HIP device.  The caller owns all buffers; the library
 *              never allocates, frees or retains them and keeps no per-call
 *              device state.
 *   Alignment  A, B and Out must be 16-byte aligned, and every row of A and
 *              B must be a whole number of 16-byte chunks (K * element size
 *              % 16 == 0); otherwise TCM_ERR_MISALIGNED.  Scale tensors need
 *              no alignment.
 *   Shapes     batch, M, N >= 0 and K >= 0.  A call with batch, M or N equal
 *              to 0 writes nothing and returns TCM_OK.  K == 0 writes zeros.
 *              Sizes whose products overflow, or negative sizes, give
 *              TCM_ERR_INVALID_SHAPE.  K > 2^20 gives TCM_ERR_UNSUPPORTED_SHAPE.
 *              Ragged M and N (not multiples of the tile) are masked.
 *   Execution  every call is asynchronous on `stream` (a hipStream_t; NULL is
 *              the default stream) and does not synchronize.  All arguments
 *              are validated on the host before any HIP call, so invalid
 *              calls return an error without touching the device.  A launch
 *              failure gives TCM_ERR_HIP.  No call falls back silently to
 *              another algorithm: an unsupported request is an error.
 *   Accuracy   element products are exact in fp32; sums are fp32.  The
 *              result r satisfies |r - exact| <= 1e-4 * sum_k |a_ik b_jk| for
 *              fp32 output, plus one bf16 ulp of the exact value for bf16
 *              output (fp32 -> bf16 is round-to-nearest-even).
 *   Threads    thread-safe: the only global state is a per-device cache of
 *              device properties filled once.
 */
#ifndef TCM_H
#define TCM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Result of every call: TCM_OK or the reason the call was refused.  This is
 * the error-or-value form of "API Card: Blackwell Pipeline (tcgen05)", Host
 * side., whose pipeline builder returns either a usable pipeline or an error
 * (one of them that a misaligned operand was given, the card's
 * alignment_unfulfilled, here TCM_ERR_MISALIGNED); unlike the card's
 * Descriptor. gates, a request the fast path cannot take is never served by
 * another algorithm but refused with one of these codes.  Ownership: a plain
 * value; nothing to free. */
typedef enum tcm_status {
    TCM_OK = 0,
    TCM_ERR_NULL_POINTER = 1,      /* a required pointer is NULL */
    TCM_ERR_INVALID_SHAPE = 2,     /* negative size or size products overflow */
    TCM_ERR_UNSUPPORTED_SHAPE = 3, /* valid but not handled (K > 2^20, MX K % 32) */
    TCM_ERR_MISALIGNED = 4,        /* pointer or row length not 16-byte aligned */
    TCM_ERR_UNSUPPORTED_DTYPE = 5, /* dtype / out_dtype pair not supported */
    TCM_ERR_NO_DEVICE = 6,         /* no HIP device, or it is not gfx950 */
    TCM_ERR_HIP = 7,               /* a HIP runtime call or kernel launch failed */
    TCM_ERR_INVALID_ARGUMENT = 8,  /* an enumeration argument outside its values */
    TCM_ERR_WORKSPACE = 9          /* the workspace is smaller than the call needs */
} tcm_status;

typedef enum tcm_dtype {
    TCM_F16 = 0,  /* IEEE binary16 */
    TCM_BF16 = 1, /* bfloat16 */
    TCM_F32 = 2,  /* IEEE binary32 */
    TCM_E4M3 = 3, /* OCP FP8 E4M3 ("FN": no infinities, max 448) */
    TCM_E8M0 = 4, /* OCP E8M0 scale: 2^(e-127), 0xFF = NaN */
    TCM_E2M1 = 5, /* OCP FP4 E2M1, two per byte, element 2t in the low four bits of
                     byte t (no infinities, no NaN, max 6) */
    TCM_E2M3 = 6, /* OCP FP6 E2M3 (bias 1, 3 mantissa bits, max 7.5), packed: see below */
    TCM_E3M2 = 7  /* OCP FP6 E3M2 (bias 3, 2 mantissa bits, max 28), packed: see below */
} tcm_dtype;

/* Arrangement of a matrix in memory: row-major (the elements of one row
 * contiguous, rows `ld` elements apart) or column-major (columns contiguous,
 * `ld` elements apart). */
typedef enum tcm_order {
    TCM_ROW_MAJOR = 0,
    TCM_COL_MAJOR = 1
} tcm_order;

/* Per-element operation of the epilogue ("API Card: Blackwell Pipeline
 * (tcgen05)", "Device side.": process_and_store(out, op)), applied in fp32 to
 * the finished value x = alpha * sum + beta * c before the rounding to the
 * output type. */
typedef enum tcm_op {
    TCM_OP_IDENTITY = 0,   /* x */
    TCM_OP_RELU = 1,       /* x if x > 0, else 0 */
    TCM_OP_GELU_TANH = 2,  /* x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) */
    TCM_OP_GELU_ERF = 3,   /* x Phi(x), Phi the standard normal distribution function */
    TCM_OP_SILU = 4        /* x / (1 + e^-x) */
} tcm_op;

/*
 * Out = A . B^T for one problem.
 *   A        M x K elements of `dtype` (TCM_F16 or TCM_BF16)
 *   B        N x K elements of `dtype`
 *   Out      M x N elements of `out_dtype` (TCM_F32 or TCM_BF16), overwritten
 * Supported pairs: (F16, F32), (F16, BF16), (BF16, F32), (BF16, BF16).
 */
tcm_status tcm_gemm_tn(const void* A, const void* B, void* Out, int64_t M, int64_t N, int64_t K,
                       tcm_dtype dtype, tcm_dtype out_dtype, void* stream);

/*
 * `batch` independent problems Out[p] = A[p] . B[p]^T, stored contiguously
 * (strides M*K, N*K, M*N elements).  Same dtypes and rules as tcm_gemm_tn;
 * the batched example of "API Card: Blackwell Pipeline (tcgen05)" (intro and
 * Descriptor.: a 128 x 256 x 64 bfloat16 tile, float accumulation, 16-byte
 * alignment) is this call with M = 128, N = 256, K = 64.
 */
tcm_status tcm_batched_gemm_tn(const void* A, const void* B, void* Out, int64_t batch, int64_t M,
                               int64_t N, int64_t K, tcm_dtype dtype, tcm_dtype out_dtype,
                               void* stream);

/*
 * Out = alpha * (A . B^T) + beta * C for one problem: the epilogue with a C
 * input ("API Card: Blackwell Pipeline (tcgen05)", "Device side.": the
 * axpby(alpha, beta, out) accessor; "mma.sync", "Accumulation, transpose and
 * alpha/beta": the scaling after the product, in a stated rounding order).
 *   A, B     as tcm_gemm_tn (dtype TCM_F16 or TCM_BF16)
 *   C        M x N elements of `c_dtype` (TCM_F16, TCM_BF16 or TCM_F32),
 *            16-byte aligned; read only when beta != 0 (then non-NULL)
 *   Out      M x N of `out_dtype` (TCM_F16, TCM_BF16 or TCM_F32), overwritten
 * The product is summed in fp32, combined as alpha * sum + beta * c in fp32,
 * and rounded once to out_dtype (round to nearest even; fp16 overflows to
 * infinity).  C may be Out itself (same pointer and dtype): every element is
 * read before it is written, by the same thread.  Partly overlapping C and
 * Out are not allowed.
 */
tcm_status tcm_gemm_tn_ex(const void* A, const void* B, const void* C, void* Out, int64_t M,
                          int64_t N, int64_t K, tcm_dtype dtype, tcm_dtype c_dtype,
                          tcm_dtype out_dtype, float alpha, float beta, void* stream);

/*
 * General form: Out = op(alpha * (A . B) + beta * C) with A the M x K matrix and B
 * the K x N matrix, each in either arrangement with a leading dimension
 * ("API Card: Blackwell Pipeline (tcgen05)", "Descriptor.": half and bfloat16
 * run in either majorness; "Host side.": global operands are declared
 * row-major or column-major with a leading dimension).
 *   A        element (i, k) at A[i*lda + k] (a_order TCM_ROW_MAJOR, lda >= K)
 *            or A[k*lda + i] (TCM_COL_MAJOR, lda >= M)
 *   B        element (k, j) at B[k*ldb + j] (b_order TCM_ROW_MAJOR, ldb >= N)
 *            or B[j*ldb + k] (TCM_COL_MAJOR, ldb >= K)
 *   C        M x N row-major of `c_dtype`, element (i, j) at C[i*ldc + j],
 *            ldc >= N; read only when beta != 0 (then non-NULL)
 *   Out      M x N row-major of `out_dtype`, element (i, j) at Out[i*ldo + j],
 *            ldo >= N; only these M x N elements are written
 * dtype TCM_F16 or TCM_BF16; c_dtype and out_dtype TCM_F16, TCM_BF16 or
 * TCM_F32.  Sums, combine and rounding as tcm_gemm_tn_ex, with `op` (a tcm_op)
 * applied in fp32 between the combine and the rounding: ReLU exactly, the
 * others from the hardware exponential and reciprocal (and, for
 * TCM_OP_GELU_ERF, the erfc approximation of Abramowitz and Stegun 7.1.26,
 * absolute error <= 1.5e-7), within 2^-20 (|x| + |op(x)|).  C may be Out itself
 * (same pointer, dtype and leading dimension).  Row-major A with
 * column-major B (lda = ldb = K, ldo = N) is tcm_gemm_tn's operation.
 * Every leading dimension must be at least 1 and at least the size named
 * above (TCM_ERR_INVALID_SHAPE), lda and ldb at most 2^21 and ldo and ldc
 * below 2^31 (TCM_ERR_UNSUPPORTED_SHAPE); an order or op outside its values
 * gives TCM_ERR_INVALID_ARGUMENT.  Alignment: A, B, Out (and C when read) 16-byte
 * aligned, lda and ldb multiples of 8 elements, and K a multiple of 8 unless
 * A is column-major and B row-major (TCM_ERR_MISALIGNED); ldo and ldc are
 * free.
 */
tcm_status tcm_gemm(const void* A, tcm_order a_order, int64_t lda, const void* B,
                    tcm_order b_order, int64_t ldb, const void* C, int64_t ldc, void* Out,
                    int64_t ldo, int64_t M, int64_t N, int64_t K, tcm_dtype dtype,
                    tcm_dtype c_dtype, tcm_dtype out_dtype, float alpha, float beta, tcm_op op,
                    void* stream);

/*
 * MXFP8 block-scaled Out = (A * SA) . (B * SB)^T.
 *   A        M x K E4M3 bytes;  B  N x K E4M3 bytes
 *   scale_A  M x (K/32) E8M0 bytes, row-major: scale_A[i][q] multiplies
 *            A[i][32q .. 32q+31]
 *   scale_B  N x (K/32) E8M0 bytes: scale_B[j][q] multiplies B[j][32q .. 32q+31]
 *   Out      M x N of `out_dtype` (TCM_F32 or TCM_BF16)
 * K must be a multiple of 32 (TCM_ERR_UNSUPPORTED_SHAPE otherwise).  A NaN
 * scale (0xFF) or element makes the affected outputs NaN.
 */
tcm_status tcm_gemm_mx_fp8(const void* A, const void* B, const void* scale_A, const void* scale_B,
                           void* Out, int64_t M, int64_t N, int64_t K, tcm_dtype out_dtype,
                           void* stream);

/*
 * MXFP4 block-scaled Out = (A * SA) . (B * SB)^T ("Hopper and Blackwell GEMM",
 * Concept, "FP8 and FP4, with block scaling": the MXFP4 row of its format
 * table, E2M1 elements with one E8M0 scale per 32).
 *   A        M x K E2M1 elements stored M x (K/2) bytes (TCM_E2M1 packing)
 *   B        N x K E2M1 elements stored N x (K/2) bytes
 *   scale_A, scale_B, Out, K, errors: as tcm_gemm_mx_fp8.
 */
tcm_status tcm_gemm_mx_fp4(const void* A, const void* B, const void* scale_A, const void* scale_B,
                           void* Out, int64_t M, int64_t N, int64_t K, tcm_dtype out_dtype,
                           void* stream);

/*
 * MXFP6 block-scaled Out = (A * SA) . (B * SB)^T (the 6-bit element formats of
 * the scaled MMA kind mxf8f6f4 named in "Hopper and Blackwell GEMM", Concept,
 * "FP8 and FP4, with block scaling"; OCP FP6 with one E8M0 scale per 32).
 *   elem_dtype  TCM_E2M3 or TCM_E3M2, for both A and B
 *   A        M x K codes packed as one little-endian bit stream per row: element
 *            t of a row in bits 6t .. 6t+5 of its bytes (four elements per
 *            three bytes), M x (3K/4) bytes
 *   B        N x K codes packed the same way, N x (3K/4) bytes
 *   scale_A, scale_B, Out, errors: as tcm_gemm_mx_fp8, except that K must be a
 *            multiple of 64 (rows of whole 16-byte pieces; TCM_ERR_MISALIGNED
 *            when K % 32 == 0 but K % 64 != 0).
 */
tcm_status tcm_gemm_mx_fp6(const void* A, const void* B, const void* scale_A, const void* scale_B,
                           void* Out, int64_t M, int64_t N, int64_t K, tcm_dtype elem_dtype,
                           tcm_dtype out_dtype, void* stream);

/*
 * MXFP8 with operands in either arrangement and leading dimensions:
 * Out = (A * SA) . (B * SB) with A the M x K and B the K x N matrix of E4M3
 * elements ("API Card: Blackwell Pipeline (tcgen05)", Descriptor.: fp8
 * types, like the 16-bit ones, reach the fast path in either majorness;
 * "Hopper and Blackwell GEMM", Concept, FP8 and FP4 with block scaling).
 *   A        a_order TCM_ROW_MAJOR: A[i * lda + k] (K contiguous, lda >= K);
 *            TCM_COL_MAJOR: A[k * lda + i] (M contiguous, lda >= M)
 *   B        b_order TCM_ROW_MAJOR: B[k * ldb + j] (N contiguous, ldb >= N);
 *            TCM_COL_MAJOR: B[j * ldb + k] (K contiguous, ldb >= K: the TN
 *            form of tcm_gemm_mx_fp8)
 *   scale_A  M x (K/32) E8M0 bytes: scale_A[i][q] multiplies a(i, 32q .. 32q+31)
 *   scale_B  N x (K/32) E8M0 bytes: scale_B[j][q] multiplies b(32q .. 32q+31, j)
 *            (the scale layout does not depend on the arrangement)
 *   Out      M x N of out_dtype (TCM_F32 or TCM_BF16), row-major, rows ldo >= N
 *            apart, overwritten
 * elem_dtype must be TCM_E4M3 (TCM_ERR_UNSUPPORTED_DTYPE otherwise).  K must
 * be a multiple of 32 (TCM_ERR_UNSUPPORTED_SHAPE); lda and ldb are multiples
 * of 16 and A, B, Out 16-byte aligned (TCM_ERR_MISALIGNED); lda, ldb <= 2^21
 * (TCM_ERR_UNSUPPORTED_SHAPE); a leading dimension below its minimum is
 * TCM_ERR_INVALID_SHAPE and an unknown order TCM_ERR_INVALID_ARGUMENT.  Sums
 * and rounding as tcm_gemm_mx_fp8, which dense TN storage (A row-major with
 * lda = K, B column-major with ldb = K, ldo = N) runs exactly.
 */
tcm_status tcm_gemm_mx(const void* A, tcm_order a_order, int64_t lda, const void* B,
                       tcm_order b_order, int64_t ldb, const void* scale_A, const void* scale_B,
                       void* Out, int64_t ldo, int64_t M, int64_t N, int64_t K,
                       tcm_dtype elem_dtype, tcm_dtype out_dtype, void* stream);

/*
 * NVFP4 Out = gA gB (A * SA) . (B * SB)^T ("Hopper and Blackwell GEMM",
 * Concept, "FP8 and FP4, with block scaling": the format table's NVFP4 row,
 * E2M1 elements with an E4M3 scale per 16 values and one FP32 scale per
 * tensor).
 *   A        M x K E2M1 elements stored M x (K/2) bytes (TCM_E2M1 packing)
 *   B        N x K E2M1 elements stored N x (K/2) bytes
 *   scale_A  M x (K/16) E4M3 bytes: scale_A[i][q] multiplies A[i][16q .. 16q+15]
 *   scale_B  N x (K/16) E4M3 bytes; both 2-byte aligned
 *   global_scale_A, global_scale_B  the per-tensor scales gA, gB
 *   Out      M x N of `out_dtype` (TCM_F16, TCM_BF16 or TCM_F32), overwritten
 * K must be a multiple of 32 (TCM_ERR_UNSUPPORTED_SHAPE).  Each element times
 * its block scale is exact in fp16; the products are summed in fp32 and
 * multiplied by the fp32 product gA gB before the one rounding to out_dtype.
 * With K a multiple of 256 and both scale tensors 16-byte aligned, a faster
 * form reads each row's scales of 256 K values at once; where such a product
 * also has enough 256 x 256 tiles to fill the device, a kernel that keeps the
 * elements 4-bit in LDS and converts them per fragment runs instead (its
 * fp32 sums run in another order, within the same bound).
 */
tcm_status tcm_gemm_nvfp4(const void* A, const void* B, const void* scale_A, const void* scale_B,
                          float global_scale_A, float global_scale_B, void* Out, int64_t M,
                          int64_t N, int64_t K, tcm_dtype out_dtype, void* stream);

/* What a call with these arguments would launch (host only: no HIP call when
 * num_cus > 0; num_cus == 0 asks the current device for its CU count). */
typedef struct tcm_plan {
    int32_t tile_m, tile_n, tile_k; /* output tile and K slice per stage */
    int32_t stages;                 /* depth of the LDS operand ring */
    int32_t threads;                /* threads per workgroup */
    int32_t stage_bytes;            /* LDS bytes of one stage (A tile + B tile) */
    int32_t lds_bytes;              /* LDS bytes of the operand ring (stages x stage_bytes);
                                       output staging and MX scale buffers add to it, within
                                       the 160 KiB of a compute unit */
    int32_t grid;                   /* workgroups launched (persistent when < tiles) */
    int64_t tiles;                  /* output tiles over all problems */
    int32_t kernel;                 /* internal kernel variant id */
} tcm_plan;

/* mx == 1 plans tcm_gemm_mx_fp8 and mx == 2 tcm_gemm_mx_fp4 (with 16-byte aligned
 * scale tensors), mx == 3 tcm_gemm_mx_fp6 (with 16-byte aligned scale tensors where
 * K % 512 == 0, else 4-byte aligned), mx == 4 tcm_gemm_nvfp4 (with 16-byte aligned scale
 * tensors), mx == 5 tcm_gemm_mx with an M- or N-major operand (dtype is then ignored);
 * other mx values are TCM_ERR_INVALID_ARGUMENT. */
tcm_status tcm_plan_gemm(int64_t batch, int64_t M, int64_t N, int64_t K, tcm_dtype dtype,
                         tcm_dtype out_dtype, int mx, int num_cus, tcm_plan* plan);

/* ---------------------------------------------------------------------------
 * The layer around the products: a projection with low-rank adapters, the
 * norm and rotation of query and key heads, a paged key-value cache and the
 * attention of one new token over it.
 *
 * The conventions above hold (asynchronous on `stream`, validated on the host,
 * no allocation).  A call that needs scratch memory takes a workspace, a device
 * buffer of at least the size its *_workspace function gives, 16-byte aligned;
 * its contents before and after a call mean nothing, and two calls may share
 * one only if one runs after the other.  Index arrays are int32 in device
 * memory.  The host cannot look at them, so the kernels check every entry
 * before they use it; what an entry outside its range means is said at each
 * call.
 * ------------------------------------------------------------------------- */

/*
 * Out[i] = X[i] . W^T + s_a (X[i] . A_a^T) . B_a^T, a = row_adapter[i]: one
 * shared projection W and, beside it, the low-rank adapter of each row's
 * request.
 *   X        M x K, rows ldx >= K elements apart;  W  N x K (dense)
 *   A        L x R x K;  B  L x N x R: L adapters of rank at most R (dense)
 *   row_adapter  M adapter numbers in any order; a row whose number is outside
 *            0 .. L-1 (-1 by custom) has the projection alone
 *   ranks    NULL, or L ranks: adapter a uses rows 0 .. ranks[a]-1 of A_a and
 *            the same columns of B_a (clipped to 0 .. R); what lies beyond them
 *            is not used and may hold anything
 *   scales   NULL (ones), or L factors s_a in fp32
 *   Out      M x N of `out_dtype`, rows ldo >= N elements apart
 * dtype TCM_F16 or TCM_BF16 (X, W, A, B); out_dtype the same or TCM_F32.  All
 * sums are fp32 and the result is rounded once.  With more than 64 rows the
 * inner product X[i] . A_a^T (times s_a) enters the second product as a sum of
 * two 16-bit values, which hold 16 bits of it (TCM_F16: 22 bits of the largest
 * of 16 consecutive ranks; fp32 outputs of TCM_BF16: three values, 24 bits),
 * whatever its size.  A row's output depends on its own adapter only: values
 * that are not finite in one adapter do not reach the rows of another.
 * R a multiple of 8, at most 128; K a multiple of 8 (TCM_ERR_MISALIGNED
 * otherwise); ldx a multiple of 8 and at most 2^21; X, W, A, B and Out 16-byte
 * aligned; Out overlaps no input.  L == 0 or R == 0 gives the projection alone.
 */
tcm_status tcm_lora_gemm_tn(const void* X, int64_t ldx, const void* W, const void* A,
                            const void* B, const int32_t* row_adapter, const int32_t* ranks,
                            const float* scales, void* Out, int64_t ldo, int64_t M, int64_t N,
                            int64_t K, int64_t L, int64_t R, tcm_dtype dtype, tcm_dtype out_dtype,
                            void* workspace, int64_t workspace_bytes, void* stream);
/* (enough also for smaller M, K and R) */
tcm_status tcm_lora_workspace(int64_t M, int64_t K, int64_t R, int64_t* bytes);

/* A view of T tokens x H heads x D elements, the D elements of a head
 * contiguous: element (t, h, d) at ptr[t * token_stride + h * head_stride + d].
 * 16-byte aligned, strides multiples of 8 elements (TCM_ERR_MISALIGNED); so a
 * slice of the heads of a fused projection is a view.  Views that a call writes
 * must not overlap themselves or each other.  Here and in a cache, the stride of a
 * dimension of one element is not looked at, nor are ldx and ldo of one row. */
typedef struct tcm_heads {
    void* ptr;
    int64_t token_stride, head_stride;
} tcm_heads;

/* A paged cache of keys and values: `pages` pages of `page_size` tokens of every
 * key-value head.  Key (p, s, h, d) lies at k[p * k_page_stride + s *
 * k_token_stride + h * k_head_stride + d], values the same way with their own
 * strides (so tokens-first and heads-first pages are both views).  dtype is
 * the type of the calls that use it, or TCM_E4M3, which stands for
 * k_scale * element and v_scale * element (the scales are not looked at
 * otherwise).  16-byte aligned, strides whole 16-byte pieces
 * (TCM_ERR_MISALIGNED); page_size at most 2^20 and token strides at most 2^25
 * elements (TCM_ERR_UNSUPPORTED_SHAPE). */
typedef struct tcm_cache {
    void* k;
    void* v;
    int64_t pages, page_size;
    int64_t k_page_stride, k_token_stride, k_head_stride;
    int64_t v_page_stride, v_token_stride, v_head_stride;
    int32_t dtype; /* a tcm_dtype */
    float k_scale, v_scale;
} tcm_cache;

/* Which elements of the rotated part of a head form a pair. */
typedef enum tcm_rope_layout {
    TCM_ROPE_HALF = 0,        /* j and j + rot_dim / 2 */
    TCM_ROPE_INTERLEAVED = 1  /* 2 j and 2 j + 1 */
} tcm_rope_layout;

/*
 * The norm and rotation of one head x (D elements):
 *   n = x w / sqrt(mean(x^2) + eps)     (norm != 0; w ones where its pointer is NULL)
 *   n = x                               (norm == 0)
 * and the pairs (n1, n2) of the first rot_dim elements turned by the angle
 * t = position * inv_freq[j]:
 *   y1 = factor (n1 cos t - n2 sin t),  y2 = factor (n2 cos t + n1 sin t);
 * the other D - rot_dim elements are n.  The angle is computed and reduced in two
 * times 64 bits and rounded once to fp32, so it is exact to 1e-7 for every int32
 * position; tables are not needed, and a scaling for long contexts is a choice of
 * inv_freq and factor.
 *   head_dim  D, a multiple of 8, at most 256 (TCM_ERR_UNSUPPORTED_SHAPE)
 *   rot_dim   even, 0 .. D (TCM_ERR_INVALID_SHAPE)
 *   positions T int32;  inv_freq  rot_dim / 2 doubles (both NULL if rot_dim == 0)
 *   q_weight, k_weight  D elements of weight_dtype: TCM_F32 or the call's dtype,
 *             16-byte aligned (TCM_ERR_MISALIGNED)
 */
typedef struct tcm_rope {
    int64_t head_dim, rot_dim;
    const int32_t* positions;
    const double* inv_freq;
    float factor;
    int32_t layout; /* a tcm_rope_layout */
    int32_t norm;
    float eps;
    const void* q_weight;
    const void* k_weight;
    int32_t weight_dtype; /* a tcm_dtype */
} tcm_rope;

/*
 * q_out = rope(norm(q)) for Hq query heads and k_out = rope(norm(k)) for Hk key
 * heads of T tokens, in one pass.  dtype TCM_F16 or TCM_BF16; computed in fp32
 * and rounded once.  Hq or Hk may be 0 (their views are then not looked at).
 * q_out may be q and k_out may be k (the same pointer and strides).
 */
tcm_status tcm_qk_norm_rope(const tcm_heads* q, const tcm_heads* k, const tcm_heads* q_out,
                            const tcm_heads* k_out, int64_t T, int64_t Hq, int64_t Hk,
                            const tcm_rope* rope, tcm_dtype dtype, void* stream);

/*
 * The same with the keys, and the values v as they are, written into a cache:
 * token t goes to slot slots[t] = page * page_size + place in the page.  A slot
 * outside 0 .. pages * page_size - 1 (-1 by custom) writes nothing to the cache;
 * its query is computed all the same.  No two tokens may have the same slot.
 * TCM_E4M3 caches take the fp32 quotient x / scale, clamped to +-448 and rounded
 * to nearest even (NaN stays NaN); scales are finite and not zero.
 */
tcm_status tcm_qk_norm_rope_cache(const tcm_heads* q, const tcm_heads* k, const tcm_heads* v,
                                  const tcm_heads* q_out, const tcm_cache* cache,
                                  const int32_t* slots, int64_t T, int64_t Hq, int64_t Hk,
                                  const tcm_rope* rope, tcm_dtype dtype, void* stream);

/*
 * Gradients of tcm_qk_norm_rope: from dq_out, dk_out (of its outputs) and its
 * inputs q, k those of the inputs, dq, dk (rounded once to dtype), and of the
 * weights, dq_weight, dk_weight (D fp32 sums over tokens and heads, overwritten;
 * NULL: not computed).  With g = w rot^T(dy) and h = x / sqrt(mean(x^2) + eps):
 *   dx = (g - h mean(g h)) / sqrt(mean(x^2) + eps),  dw = sum rot^T(dy) h.
 * Sums run in a fixed order: the same call gives the same bits.  dq may be
 * dq_out and dk dk_out.  T == 0 gives zero weight gradients.
 */
tcm_status tcm_qk_norm_rope_bwd(const tcm_heads* dq_out, const tcm_heads* dk_out,
                                const tcm_heads* q, const tcm_heads* k, const tcm_heads* dq,
                                const tcm_heads* dk, float* dq_weight, float* dk_weight, int64_t T,
                                int64_t Hq, int64_t Hk, const tcm_rope* rope, tcm_dtype dtype,
                                void* workspace, int64_t workspace_bytes, void* stream);
tcm_status tcm_qk_norm_rope_bwd_workspace(int64_t head_dim, int64_t* bytes);

/*
 * Attention of one new token per sequence over a paged cache: for sequence b
 * and query head h (key-value head h / (Hq / Hk)),
 *   out = sum_j p_j v_j,  p = softmax_j(scale * q . k_j),
 * j over the keys max(0, n - window) .. n - 1 of the sequence (window == 0: all),
 * n = lengths[b].  Key j lies in page block_table[b * table_stride + j / page_size]
 * at place j % page_size.
 *   q, out   views of B tokens x Hq heads x D; out may be q
 *   block_table  B rows of table_stride entries; an entry outside 0 .. pages-1
 *            is a hole, whose keys are not attended
 *   lengths  B int32, clipped to 0 .. min(max_len, table_stride * page_size)
 *   lse      NULL, or B x Hq fp32 (dense): log sum_j exp(scale * q . k_j)
 *   max_len  an upper bound of the lengths, which the split over the length
 *            goes by (a graph captured with it serves every length up to it)
 * A sequence without keys gives out = 0 and lse = -infinity.  Cache memory
 * that holds no attended key is not used and may hold anything.
 * dtype (q, out) TCM_F16 or TCM_BF16, the cache's dtype the same or TCM_E4M3.  Scores,
 * softmax and sums in fp32; the probabilities enter the second product as the
 * sum of two values of dtype (16 bits of them for TCM_BF16, 22 for TCM_F16, of
 * which those 2^-40 of a row's largest are the last).  D a multiple of 8 (16 for TCM_E4M3 caches), at most 256; Hq a multiple of
 * Hk; B and Hq at most 65535.
 */
tcm_status tcm_paged_attention(const tcm_heads* q, const tcm_cache* cache,
                               const int32_t* block_table, int64_t table_stride,
                               const int32_t* lengths, int64_t max_len, const tcm_heads* out,
                               float* lse, int64_t B, int64_t Hq, int64_t Hk, int64_t D,
                               float scale, int64_t window, tcm_dtype dtype, void* workspace,
                               int64_t workspace_bytes, void* stream);
/* (enough also for smaller B and max_len and for every window) */
tcm_status tcm_paged_attention_workspace(int64_t B, int64_t Hq, int64_t Hk, int64_t D,
                                         int64_t max_len, int64_t* bytes);

/* Static, human-readable name of a status code, the counterpart of the error
 * string lookup of "API Card: Blackwell Pipeline (tcgen05)", Host side.
 * (which names the card's error values, alignment_unfulfilled among them).
 * Codes outside the enumeration give "TCM_ERR_UNKNOWN: unknown status code".  The string is
 * static and owned by the library (never NULL, never freed by the caller);
 * the call touches no device and is thread-safe. */
const char* tcm_status_string(tcm_status s);

#ifdef __cplusplus
}
#endif

#endif /* TCM_H */
