/*
 * sgemm.h -- C ABI of the GB300 (sm_103a) single-precision GEMM library.
 *
 * Operation (the definition on the page "Deep dive into the sgemmNN
 * algorithm" (lazypool blog), section "Why SGEMM matters"; argument list in
 * the style of the sgemmNN kernel signature on the same page, section
 * "The whole kernel"):
 *
 *     C <- alpha * A * B + beta * C
 *
 * with A an M x K, B a K x N and C an M x N matrix of 32-bit floats, all
 * ROW-MAJOR with leading dimensions (element strides between rows):
 *
 *     A[i][p] = A[i*lda + p],  B[p][j] = B[p*ldb + j],  C[i][j] = C[i*ldc + j]
 *
 * (row-major as in the naive kernel of page m.lqnn.cn/news/94381, section
 * 1.1).  Accumulation is in FP32 on the GPU; the summation order is the
 * library's and is fixed per kernel variant, so repeated calls with the same
 * inputs and the same variant give bit-identical results.
 *
 * Conventions (BLAS, where the pages are silent):
 *   - beta == 0: C is output only and is never read (NaN/Inf in C do not
 *     propagate).
 *   - alpha == 0 or K == 0: A and B are not read (may be NULL); C <- beta*C.
 *   - M == 0 or N == 0: nothing is done; every pointer may be NULL.
 *   - Cells outside the M x K, K x N, M x N windows (columns K..lda-1 of A,
 *     N..ldb-1 of B, N..ldc-1 of C) are never read or written.
 *   - Any 4-byte-aligned pointer and any leading dimension is accepted.  An
 *     operand the TMA cannot read as stored (not 16-byte aligned, or its
 *     leading dimension -- or batch stride -- not a multiple of 4) is either
 *     read with scalar loads by the generic variant or first copied
 *     transposed, on the GPU, into the handle's re-layout workspace, which
 *     the TMA kernels then read (whichever the library estimates faster;
 *     see sgemm_relayout_t).  Never an error, never a CPU path.
 *
 * Column-major (BLAS / Fortran order) callers: a column-major m x n matrix
 * with leading dimension ld is the row-major n x m matrix of its transpose,
 * so the column-major product C = op(A) * op(B) is the row-major product
 * C^T = op(B)^T * op(A)^T: call sgemm_run_ex with the operands swapped
 * together with their trans flags and leading dimensions (B, transB, ldb
 * first; A, transA, lda second) and M and N swapped.
 *
 * Memory and streams: all matrix pointers are DEVICE pointers owned by the
 * caller.  sgemm_run never allocates and never synchronizes: it validates
 * its arguments on the host, enqueues kernels on `stream` (a cudaStream_t
 * cast to void*, NULL for the legacy default stream) and returns.  The
 * returned status covers only what is known at enqueue time; a fault found
 * later by a kernel is reported by sgemm_get_device_status.
 *
 * Threading: one handle may be used from one host thread at a time, and its
 * calls must be ordered on the GPU (one stream, or streams ordered by
 * events): calls of the same handle share its stream-K and re-layout
 * workspaces.  Use one handle per concurrently running stream.
 *
 * Every function returns an sgemm_status_t value (as int) unless noted.
 */
#ifndef SGEMM_H
#define SGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sgemm_ctx *sgemm_handle_t;

typedef enum {
    SGEMM_OK = 0,
    SGEMM_ERR_NULL = 1,               /* a required pointer argument is NULL          */
    SGEMM_ERR_INVALID_VALUE = 2,      /* negative size, ld below its minimum, bad enum */
    SGEMM_ERR_ALIAS = 3,              /* C overlaps A or B                             */
    SGEMM_ERR_BAD_HANDLE = 4,         /* not a live handle (never created, destroyed)  */
    SGEMM_ERR_UNSUPPORTED_DEVICE = 5, /* current device is not compute capability 10.3 */
    SGEMM_ERR_LAUNCH = 6,             /* the kernel launch was rejected                */
    SGEMM_ERR_CUDA = 7,               /* another CUDA runtime error                    */
    SGEMM_ERR_DEVICE_TIMEOUT = 8,     /* a kernel gave up a bounded wait (device side) */
    SGEMM_ERR_WRONG_DEVICE = 9,       /* current device differs from the handle's      */
    SGEMM_ERR_SCRATCH_TOO_SMALL = 10, /* sgemm_run_noalloc: problem exceeds its scratch */
    SGEMM_ERR_DEVICE_CHECK = 11       /* a device-side index check failed (builds with
                                         -DSGEMM_DEVICE_CHECKS only)                    */
} sgemm_status_t;

/* Kernel variants.  SGEMM_VARIANT_AUTO lets sgemm_run choose from the shape
 * and the alignment of the operands; the others pin one variant (for tests
 * and measurements).  A pinned TMA variant on an operand the TMA cannot read
 * as stored runs on its transposed copy (the re-layout workspace), or, when
 * the re-layout is off or the copy does not fit, is replaced by the generic
 * variant for that call. */
typedef enum {
    SGEMM_VARIANT_AUTO = 0,
    SGEMM_VARIANT_TMA_128x256 = 1,   /* TMA-fed SIMT, 128 x 256 CTA tile, 8 x 16 per thread */
    SGEMM_VARIANT_TMA_128x128 = 2,   /* TMA-fed SIMT, 128 x 128 CTA tile, 8 x 8 per thread  */
    SGEMM_VARIANT_TMA_64x64 = 3,     /* TMA-fed SIMT, 64 x 64 CTA tile, 8 x 4 per thread    */
    SGEMM_VARIANT_TMA_64x64_SPLITK = 4, /* 64 x 64 tiles, stream-K over all tiles, fixed-order sum */
    SGEMM_VARIANT_GENERIC = 5,       /* scalar loads, any alignment, 64 x 64 CTA tile       */
    SGEMM_VARIANT_SCALE = 6,         /* reported only: the C <- beta*C quick path ran       */
    SGEMM_VARIANT_TC_3XTF32 = 7,     /* tensor cores (tcgen05, TMEM), 3xTF32 split precision,
                                        128 x 256 CTA tile; FP32 inputs, outputs, tolerance   */
    SGEMM_VARIANT_TC_3XTF32_PAIR = 8,/* as TC_3XTF32 on CTA pairs (cta_group::2): 256 x 256
                                        tile per cluster of two CTAs                          */
    SGEMM_VARIANT_TC_F16_PAIR = 9,   /* sgemm_run_mixed only: BF16 / FP16 A and B on the tensor
                                        cores (kind::f16), FP32 accumulation, CTA pairs       */
    SGEMM_VARIANT_GENERIC_F16 = 10,  /* sgemm_run_mixed only: the generic variant on 16-bit
                                        inputs (any alignment)                                */
    SGEMM_VARIANT_TMA_256x128 = 11,  /* TMA-fed SIMT, 256 x 128 CTA tile, 16 warps, 8 x 8 per
                                        thread (fastest on large problems)                    */
    SGEMM_VARIANT_TC_I8 = 12,        /* sgemm_run_int8, sgemm_run_int8_experts only: int8 operands
                                        as exact FP16 on the tensor cores, int32 sums         */
    SGEMM_VARIANT_GENERIC_I8 = 13,   /* the same calls: any layout and alignment, CUDA cores  */
    SGEMM_VARIANT_FEW_I8 = 14,       /* sgemm_run_int8 only: up to 8 rows of A, CUDA cores, B
                                        stored N x K on any alignment                         */
    SGEMM_VARIANT_TC_F4 = 15,        /* sgemm_run_fp4 only: tensor cores with block scales, 128
                                        channels x 16 to 128 tokens a CTA, K split over clusters */
    SGEMM_VARIANT_TC_F4_PAIR = 16,   /* sgemm_run_fp4 only: the same on CTA pairs, 256 x 256     */
    SGEMM_VARIANT_GENERIC_F4 = 17,   /* sgemm_run_fp4 only: any alignment, CUDA cores            */
    SGEMM_VARIANT_COUNT_ = 18
    /* sgemm_run_ex: the TMA variants serve every (transA, transB) and any
     * batch up to 65535 when A and B are 16-byte aligned and lda, ldb (and,
     * for batch > 1, strideA, strideB) are multiples of 4, and operands that
     * are not through their transposed copies (above); otherwise the generic
     * variant runs.  The tensor-core variants serve every layout
     * and batches of up to 256 products (one launch per product): they read
     * A stored M x K and B stored K x N, and an operand stored transposed is
     * first copied into that layout in the re-layout workspace (one launch
     * per copy; see sgemm_relayout_t).  Where that cannot be done (a larger
     * batch, re-layout off, copies larger than the workspace) a pinned
     * tensor-core variant acts as AUTO. */
} sgemm_variant_t;

/* Arithmetic used by SGEMM_VARIANT_AUTO.  Both modes meet the same FP32
 * contract (max |C - C_exact| within 1e-3 for K <= 1024 and 1e-2 for K <= 8192
 * on U[-1,1) data).  SGEMM_MATH_FP32 (the default) runs FP32 FMAs on the CUDA
 * cores.  SGEMM_MATH_3XTF32 lets the library use the tensor cores with the
 * 3xTF32 split-precision method (A*B = A_hi*B_hi + A_hi*B_lo + A_lo*B_hi) for
 * problems large enough to profit; its rounding errors are larger than the
 * FP32 path's (about 5x at K = 8192) but still inside the contract.  In this
 * mode SGEMM_VARIANT_AUTO takes SGEMM_VARIANT_TC_3XTF32_PAIR when there are at
 * least SMs/4 tiles of 256 x 256 and K >= 256 and the tensor-core kernels can
 * serve the call (see sgemm_variant_t), and the FP32 kernels otherwise. */
typedef enum {
    SGEMM_MATH_FP32 = 0,
    SGEMM_MATH_3XTF32 = 1
} sgemm_math_mode_t;

/* Operand re-layout of the FP32 SIMT path (sgemm_run, sgemm_run_ex, any
 * batch; the tensor-core variants' copies into the NN
 * layout use the same workspace and are off with SGEMM_RELAYOUT_OFF).  A
 * strided batch is copied matrix by matrix (an operand with batch stride 0
 * once), each copy in its own slot of the workspace.  On GB300 the SIMT kernel's main loop is
 * fastest with A stored K x M and B stored K x N (transA = 1, transB = 0:
 * one 16-byte shared-memory load then gives one k of four rows of A).  The
 * library may therefore first copy A stored M x K, or B stored N x K,
 * transposed into the handle's re-layout workspace (an HBM-bound pass,
 * about 0.6 % of the time of an 8192^3 product) and run the GEMM on the
 * copy.  Every layout forms each product in ascending k with one rounding
 * per FMA, so with the same tile variant and the same stream-K plan the
 * result is bit-identical to the call without re-layout.
 * An operand the TMA cannot read as stored (see the conventions above) is
 * copied transposed whatever its stored layout, and the other operand as
 * the estimate prefers; the generic variant runs instead when its estimate
 * is lower (small problems: about 9 us of fixed cost against the copies'
 * launches).
 *   SGEMM_RELAYOUT_AUTO (default): when the library's time estimate of the
 *     copies plus the faster kernel beats the kernel on the operands as
 *     stored by at least 1 % and the copies fit in the workspace (an
 *     operand the TMA cannot read: when they fit and beat the generic
 *     variant);
 *   SGEMM_RELAYOUT_OFF: never (an operand the TMA cannot read: the generic
 *     variant);
 *   SGEMM_RELAYOUT_ALWAYS: whenever the copies that reach transA = 1,
 *     transB = 0 fit in the workspace (tests, measurements). */
typedef enum {
    SGEMM_RELAYOUT_AUTO = 0,
    SGEMM_RELAYOUT_OFF = 1,
    SGEMM_RELAYOUT_ALWAYS = 2
} sgemm_relayout_t;

/* Formats of rows in 4-bit floating point (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 with
 * a sign) with a scale for every block of consecutive elements of a row. */
typedef enum {
    SGEMM_FP4_MX = 0,   /* blocks of 32, scales E8M0: 2^(byte - 127), 255 a NaN                */
    SGEMM_FP4_NV = 1    /* blocks of 16, scales E4M3 (>= 0), and one FP32 scale a row          */
} sgemm_fp4_t;

/* Element type of A and B for sgemm_run_mixed (BF16 and FP16; C is always
 * FP32), of the rows that the quantization and expert calls read and write,
 * and of the int8 products' C (any of the three). */
typedef enum {
    SGEMM_IN_F32 = 0,   /* FP32 (not for sgemm_run_mixed) */
    SGEMM_IN_BF16 = 1,  /* bfloat16: 1 sign, 8 exponent, 7 fraction bits */
    SGEMM_IN_F16 = 2    /* IEEE binary16 */
} sgemm_input_t;

/* Create a handle bound to the CURRENT CUDA device.  Requires compute
 * capability 10.3 (GB300); otherwise returns SGEMM_ERR_UNSUPPORTED_DEVICE and
 * sets *out to NULL.  Allocates the handle's device-side status word, its
 * stream-K workspace (48 MiB) and arrival counters (zeroed), and its operand
 * re-layout workspace (512 MiB: the transposes of an 8192 x 8192 A and B;
 * if that allocation fails the handle is created without it and never
 * re-lays out), and sets the kernels' shared-memory limits.  `out` must be
 * non-NULL (else SGEMM_ERR_NULL). */
int sgemm_create(sgemm_handle_t *out);

/* C <- alpha*A*B + beta*C, enqueued on `stream`; see the conventions above.
 * Argument checks, in order: handle (SGEMM_ERR_BAD_HANDLE), current device
 * (SGEMM_ERR_WRONG_DEVICE), then the rules of sgemm_check_args.  On any
 * error nothing is enqueued and C is unchanged. */
int sgemm_run(sgemm_handle_t h, int M, int N, int K, float alpha,
              const float *A, int lda, const float *B, int ldb,
              float beta, float *C, int ldc, void *stream);

/* The general form: C_b <- alpha * op(A_b) * op(B_b) + beta * C_b for b = 0 ..
 * batch-1, where op(X) = X (trans = 0) or X^T (trans = 1), op(A) is M x K,
 * op(B) is K x N, and matrix b of each operand starts `stride` elements after
 * matrix b-1 (X_b = X + b*strideX).  Row-major storage as above: A is stored
 * M x K (lda >= max(1, K)) when transA = 0 and K x M (lda >= max(1, M)) when
 * transA = 1; B is stored K x N (ldb >= max(1, N)) when transB = 0 and N x K
 * (ldb >= max(1, K)) when transB = 1.  `sgemm_run` is the case transA = transB
 * = 0, batch = 1.  Strides must be >= 0; with batch > 1 the C matrices must not
 * overlap one another (strideC at least the extent of one C window), else
 * SGEMM_ERR_INVALID_VALUE.  batch == 0 is a no-op.  The pages' sgemmNN kernel
 * (page "Deep dive into the sgemmNN algorithm") is the NN case; the transposed
 * and batched forms are the BLAS / cuBLAS conventions the pages' batched call
 * (page "GPU-accelerated matrix computation optimisation and CUDA programming
 * practice", section 4.2) uses. */
int sgemm_run_ex(sgemm_handle_t h, int transA, int transB, int M, int N, int K, float alpha,
                 const float *A, int lda, long long strideA, const float *B, int ldb, long long strideB,
                 float beta, float *C, int ldc, long long strideC, int batch, void *stream);

/* Host-only validation of sgemm_run_ex's arguments (same rules, no CUDA call). */
int sgemm_check_args_ex(int transA, int transB, int M, int N, int K, float alpha, const float *A, int lda,
                        long long strideA, const float *B, int ldb, long long strideB, float beta,
                        const float *C, int ldc, long long strideC, int batch);

/* Mixed precision: C <- alpha * op(A) * op(B) + beta * C with A and B holding
 * 16-bit values (`in_type`: SGEMM_IN_BF16 or SGEMM_IN_F16; 2 bytes per element,
 * leading dimensions in elements) and C in FP32.  op and the stored shapes as
 * in sgemm_run_ex (batch 1).  Every product of two 16-bit values is exact in
 * FP32; the products are summed in FP32 (on the tensor cores, whose FP32
 * accumulation is not round-to-nearest), then alpha, beta and C as in
 * sgemm_run.  Error contract: max |C - C_exact| within 1e-3 for K <= 1024
 * and 1e-2 for K <= 8192 on inputs of magnitude <= 1, where C_exact is the
 * exact result for the 16-bit inputs as given (the caller's rounding to 16 bits
 * is not part of it).  Page "GPU-accelerated matrix computation optimisation
 * and CUDA programming practice", section 4.1, uses this split (16-bit inputs,
 * FP32 accumulation) through a library call; here it is a kernel of this
 * library.  Runs SGEMM_VARIANT_TC_F16_PAIR when A and B are 16-byte aligned and
 * lda, ldb are multiples of 8, else SGEMM_VARIANT_GENERIC_F16 (a pinned
 * GENERIC variant also selects it).  Errors as sgemm_run_ex, plus
 * SGEMM_ERR_INVALID_VALUE for an unknown in_type. */
int sgemm_run_mixed(sgemm_handle_t h, int in_type, int transA, int transB, int M, int N, int K, float alpha,
                    const void *A, int lda, const void *B, int ldb, float beta, float *C, int ldc, void *stream);

/* Host-only validation of sgemm_run_mixed's arguments (same rules, no CUDA call). */
int sgemm_check_args_mixed(int in_type, int transA, int transB, int M, int N, int K, float alpha, const void *A,
                           int lda, const void *B, int ldb, float beta, const float *C, int ldc);

/* ---- 8-bit integer products ------------------------------------------------
 *
 *     C[i][j] = scaleA[i] * scaleB[j] * sum_p A[i][p] * op(B)[p][j] + bias[j]
 *
 * with int8 A (M x K, M tokens) and B, one FP32 scale a row of A (a token) and
 * one a column of op(B) (a channel), an optional FP32 bias a channel (NULL:
 * none), and C of type `out_type` (an sgemm_input_t).  B is stored N x K
 * (transB = 1, a linear layer's weights; fastest) or K x N (transB = 0), all
 * row-major, leading dimensions in elements.  The sum is exact (32-bit
 * integers; K <= 131071, the longest that cannot overflow, else
 * SGEMM_ERR_INVALID_VALUE) and float(sum) * scaleB * scaleA + bias is rounded
 * to C's type once, so results do not depend on the variant or on how the work
 * was split.  All 256 values of an int8 are taken as they are.  C is output
 * only.  Bytes between the rows of A and of B may be read together with their
 * neighbours, and do not matter.  K == 0 gives C = bias.  FP16 results beyond 65504 become infinite.
 *
 * A may have any alignment and leading dimension.  B is read in place when
 * transB = 1, B is 16-byte aligned and ldb is a multiple of 16 (in the expert
 * form strideB too); otherwise it is first copied into the re-layout workspace
 * (sgemm_last_relayout then reports bit 1; calls of up to 8 rows of A may read
 * it in place on any alignment).  A's rows are copied there where they
 * do not start on 16-byte boundaries and, by the calls with many rows, expanded
 * to FP16 (2 bytes an element), in several passes where they do not fit.  One
 * launch makes all copies of a pass, and one multiplies: 1 launch where nothing
 * is copied, else 2 a pass (sgemm_last_launches); sgemm_last_variant
 * reports the CTAs that share a tile's K range.  Without the workspace where a
 * copy is needed, with SGEMM_RELAYOUT_OFF where B would be copied, where the
 * copies do not fit, or with SGEMM_VARIANT_GENERIC or _GENERIC_I8 pinned, the
 * generic kernel runs.  Otherwise as sgemm_run: no allocation, no
 * synchronization, device pointers, one handle per concurrently running stream.
 *
 * Checks, in order: handle, device, then (sgemm_check_args_int8)
 * SGEMM_ERR_INVALID_VALUE for an unknown out_type or transB, a negative size, M or
 * N above 2^30, K above 131071, lda < max(1, K), ldb or ldc below its minimum; nothing is done
 * when M == 0 or N == 0; SGEMM_ERR_NULL if C, scaleA or scaleB (or A or B while
 * K > 0) is NULL; SGEMM_ERR_INVALID_VALUE if C, a scale array or the bias is
 * not aligned to its element size; SGEMM_ERR_ALIAS if C overlaps an input. */
int sgemm_run_int8(sgemm_handle_t h, int transB, int out_type, int M, int N, int K, const int8_t *A, int lda,
                   const float *scaleA, const int8_t *B, int ldb, const float *scaleB, const float *bias, void *C,
                   int ldc, void *stream);

/* Host-only validation of sgemm_run_int8's arguments (same rules, no CUDA call). */
int sgemm_check_args_int8(int transB, int out_type, int M, int N, int K, const int8_t *A, int lda,
                          const float *scaleA, const int8_t *B, int ldb, const float *scaleB, const float *bias,
                          const void *C, int ldc);

/* The same product over rows sorted by expert: rows offsets[e] .. offsets[e+1]-1
 * of A and C use B_e = B + e*strideB, scaleB + e*N and bias + e*N (e = 0 ..
 * experts-1; scaleB and bias hold experts*N values).  `offsets` (experts + 1
 * ints) is in DEVICE memory, as sgemm_expert_sort writes it: the call needs no
 * host copy of it.  Rows before offsets[0] or from offsets[experts] on belong
 * to no expert: their A is not used and their C is not written.  Offsets
 * outside [0, rows] or out of order are taken as the nearest bounds that are
 * in order, so no access leaves the buffers.  experts is 1 .. 1024; strideB
 * (elements) >= 0, 0 giving every expert the same B.  Checks as above, plus
 * SGEMM_ERR_NULL for NULL offsets. */
int sgemm_run_int8_experts(sgemm_handle_t h, int transB, int out_type, int experts, int rows, int N, int K,
                           const int *offsets, const int8_t *A, int lda, const float *scaleA, const int8_t *B,
                           int ldb, long long strideB, const float *scaleB, const float *bias, void *C, int ldc,
                           void *stream);

/* Host-only validation of sgemm_run_int8_experts's arguments. */
int sgemm_check_args_int8_experts(int transB, int out_type, int experts, int rows, int N, int K, const int *offsets,
                                  const int8_t *A, int lda, const float *scaleA, const int8_t *B, int ldb,
                                  long long strideB, const float *scaleB, const float *bias, const void *C, int ldc);

/* Rows to 8-bit integers: for each row i of X (M x K, of `type`), with m the
 * largest |X[i][p]|,
 *     scale[i] = m / 127,    Q[i][p] = rint(X[i][p] * (127 / m))
 * (each operation correctly rounded in FP32, ties to even), so that
 * Q[i][p] * scale[i] is X[i][p] to within scale[i] / 2 and a rounding.  A row
 * with m < 127 * 2^-126 (all zeros among them) gives Q = 0, scale = 0; a row
 * with an infinity or a NaN gives Q = 0, scale = NaN, so that every product
 * with it is NaN.  K == 0 gives scales of 0.  Checks: handle, device,
 * SGEMM_ERR_INVALID_VALUE (unknown type, negative size, K above 2^30, leading
 * dimension below max(1, K)), M == 0 does nothing, SGEMM_ERR_NULL,
 * SGEMM_ERR_INVALID_VALUE (a pointer not aligned to its element size),
 * SGEMM_ERR_ALIAS (any two of the three overlap). */
int sgemm_quantize_rows(sgemm_handle_t h, int type, int M, int K, const void *X, int ldx, int8_t *Q, int ldq,
                        float *scale, void *stream);

/* ---- rows in 4-bit floating point --------------------------------------------
 *
 * An element is row[i] * s[i][b] * q[i][p], b the block of p (sgemm_fp4_t; 32 or 16
 * elements, the last of a row shorter where they do not divide K).
 *   Q: two elements a byte, the even one in the low half; rows ldq >= ceil(K / 2)
 *     BYTES apart, any alignment (multiples of 16 let the products read them in place).
 *     The half byte behind an odd K is 0.
 *   S: the scales in tiles of 128 rows x 4 blocks, sgemm_fp4_scale_bytes bytes, 16-byte
 *     aligned.  With words = ceil(ceil(K / block) / 4), the scale of row i and block b is
 *       S[((i / 128) * words + b / 4) * 512 + (i % 32) * 16 + (i / 32) % 4 * 4 + b % 4].
 *     Scales of blocks behind a row's last within its last word are 0; those of rows
 *     behind the last are not written and may hold anything.
 *   row: one FP32 a row; required with SGEMM_FP4_NV, with SGEMM_FP4_MX NULL for ones.
 * Buffers made elsewhere have to be laid out in the same way, the zeros included.
 *
 * sgemm_quantize_fp4 makes them from rows X of `type`.  Each step is correctly rounded
 * in FP32, ties to even; m is the row's largest magnitude, m_b a block's:
 *   MX: s = 2^e with e = floor(log2 m_b) - 2, at least -127 (a block of zeros: -127);
 *       q = X / s to the nearest of the values, magnitudes above 6 to 6;
 *       row (NULL allowed) = 1.  A block with an infinity or a NaN gets s = NaN, q = 0.
 *   NV: row = m / 2688;  s = E4M3(m_b * (448 / m));  q = X * ((2688 / m) / s) likewise
 *       (s = 0: q = 0; the quotient, which can pass FP32's range where m < 2688 * 2^-118, as
 *       with an exponent without bounds).  A row with m < 2688 * 2^-126 (all zeros among them)
 *       gets row = 0, s = 0, q = 0; a row with an infinity or a NaN row = NaN, s = 0, q = 0.
 * Every product with a NaN scale is NaN.
 * sgemm_dequantize_fp4 gives Y = row * s * q, rounded to FP32 and then to `type`.
 *
 * Checks, in order: handle, device, SGEMM_ERR_INVALID_VALUE (unknown type or format,
 * negative size, M or K above 2^30, a leading dimension below its minimum), nothing
 * is done when M == 0 or K == 0, SGEMM_ERR_NULL, SGEMM_ERR_INVALID_VALUE (alignment),
 * SGEMM_ERR_ALIAS (an output overlaps another buffer). */
int sgemm_quantize_fp4(sgemm_handle_t h, int type, int format, int M, int K, const void *X, int ldx, uint8_t *Q,
                       int ldq, uint8_t *S, float *row, void *stream);
int sgemm_dequantize_fp4(sgemm_handle_t h, int type, int format, int M, int K, const uint8_t *Q, int ldq,
                         const uint8_t *S, const float *row, void *Y, int ldy, void *stream);

/* Bytes of the scales of `rows` rows of K elements: whole tiles.  -1 for an unknown
 * format or a size outside [0, 2^30].  Host only. */
int64_t sgemm_fp4_scale_bytes(int format, int rows, int K);

/*     C[i][j] = rowA[i] * rowB[j] * sum_p (sA q_A)[i][p] * (sB q_B)[j][p] + bias[j]
 *
 * for A (M tokens) and B (N channels, stored N x K) in the same 4-bit format, an optional
 * FP32 bias a channel, and C (M x N) of type `out_type`.  lda and ldb in bytes, ldc in
 * elements.  Products are exact, summed in FP32 by the tensor cores (not
 * round-to-nearest, in an order that depends on the variant and the split; the same
 * call gives the same bits every time); sum * rowB * rowA + bias is rounded to C's type.
 * With SGEMM_FP4_MX either row scale may be NULL.  C is output only; K == 0 gives the bias.
 *
 * A and B are read in place where they are 16-byte aligned with rows multiples
 * of 16 bytes apart, and otherwise first copied into the re-layout workspace
 * (sgemm_last_relayout: bit 0 A, bit 1 B; one more launch for both).  Where the
 * copies do not fit or SGEMM_RELAYOUT_OFF forbids them, or with SGEMM_VARIANT_GENERIC
 * or _GENERIC_F4 pinned, the generic kernel runs.  SGEMM_VARIANT_TC_F4 and _TC_F4_PAIR may be
 * pinned; then they run at any size where the generic kernel need not.
 * sgemm_last_variant also reports the CTAs that share a tile's K range.
 * Checks as for the 4-bit rows, nothing done when M == 0 or N == 0. */
int sgemm_run_fp4(sgemm_handle_t h, int format, int out_type, int M, int N, int K, const uint8_t *A, int lda,
                  const uint8_t *SA, const float *rowA, const uint8_t *B, int ldb, const uint8_t *SB,
                  const float *rowB, const float *bias, void *C, int ldc, void *stream);

/* Host-only validation of sgemm_run_fp4's arguments (same rules, no CUDA call). */
int sgemm_check_args_fp4(int format, int out_type, int M, int N, int K, const uint8_t *A, int lda,
                         const uint8_t *SA, const float *rowA, const uint8_t *B, int ldb, const uint8_t *SB,
                         const float *rowB, const float *bias, const void *C, int ldc);

/* ---- RMS norm ------------------------------------------------------------------
 *
 * Rows X (M x K) of `type`, weights (K) of the same type, eps >= 0:
 *   H = X + R, rounded to `type`       (R NULL: H stands for X itself, and is written
 *                                       where it is not NULL)
 *   r = 1 / sqrt(sum_p H_p^2 / K + eps)
 *   sgemm_rms_norm        Y = (H * r) * weight, and r to rstd (NULL: not wanted)
 *   sgemm_rms_norm_int8   v = H * weight, m = max |v|:  Q = rint(v * (127 / m)),
 *                         scale = m * r / 127
 *   sgemm_rms_norm_fp4    v as by sgemm_quantize_fp4, the row scales times r (required
 *                         with either format: with MX they are r)
 * The quantized forms are the input of sgemm_run_int8 and sgemm_run_fp4; what v rounds to
 * does not depend on r, so the integers and codes are the same whatever the order of
 * a sum.  Special rows as by sgemm_quantize_rows and sgemm_quantize_fp4.  Sums are in FP32,
 * in a fixed order; a row whose sum of squares overflows FP32 has r = 0.  With eps = 0 a row
 * whose sum of squares is 0 has r = infinity: of a row of zeros the Y of sgemm_rms_norm (and
 * its gradient) is NaN, the quantized forms make zeros with row scales of 0.
 *
 * sgemm_rms_norm_grad, from dY, the gradient dH that reaches H from elsewhere (the
 * residual's further way; NULL: none), H and rstd:
 *   dX = r * (weight * dY) - H * r^3 / K * sum_p (weight dY H)_p + dH   (X's gradient and R's)
 *   dweight_p = sum_i (dY * H * r)_ip                                    (FP32; M == 0: zeros)
 * It adds up dweight in the handle's workspace: K up to 12582912.
 *
 * H may be X or R in place (same address, same leading dimension), and dX dH.
 * Checks, in order: handle, device, SGEMM_ERR_INVALID_VALUE (sizes, type, format, leading
 * dimensions, eps; K above 2^30, with 4 bits M too), nothing is done when M == 0 or K == 0,
 * SGEMM_ERR_NULL (R without H among them), SGEMM_ERR_INVALID_VALUE (alignment to
 * the element size, S to 16 bytes), SGEMM_ERR_ALIAS. */
int sgemm_rms_norm(sgemm_handle_t h, int type, int M, int K, const void *X, int ldx, const void *R, int ldr,
                   const void *weight, float eps, void *H, int ldh, void *Y, int ldy, float *rstd, void *stream);
int sgemm_rms_norm_int8(sgemm_handle_t h, int type, int M, int K, const void *X, int ldx, const void *R, int ldr,
                        const void *weight, float eps, void *H, int ldh, int8_t *Q, int ldq, float *scale,
                        void *stream);
int sgemm_rms_norm_fp4(sgemm_handle_t h, int type, int format, int M, int K, const void *X, int ldx, const void *R,
                       int ldr, const void *weight, float eps, void *H, int ldh, uint8_t *Q, int ldq, uint8_t *S,
                       float *row, void *stream);
int sgemm_rms_norm_grad(sgemm_handle_t h, int type, int M, int K, const void *dY, int lddy, const void *dH, int lddh,
                        const void *H, int ldh, const void *weight, const float *rstd, void *dX, int lddx,
                        float *dweight, void *stream);

/* ---- tokens to their experts and back ----------------------------------------
 *
 * A router gives each of `tokens` tokens `choices` experts: ids[t*choices + j].
 * Slot s = t*choices + j is choice j of token t; a slot whose id is outside
 * [0, experts) is dropped (a capacity limit's way to say so).
 *
 * sgemm_expert_sort orders the slots by expert, slots of one expert in
 * ascending order: offsets[e] is the first row of expert e and
 * offsets[experts] the number of slots kept; rows[s] the row of slot s, -1 for
 * a dropped one; source[r] the slot of row r, -1 for the rows from
 * offsets[experts] on.  (experts + 1, tokens*choices and tokens*choices ints.)
 * The order is the same on every call.  experts is 1 .. 1024 and
 * tokens*choices < 2^31 (sort: at most 2^14 * floor(12582912 / experts) slots, 201
 * million with 1024 experts -- the counts that its workspace holds -- else
 * SGEMM_ERR_INVALID_VALUE).
 *
 * The other calls move rows of `width` elements of `type`; the tokens' side has
 * `tokens` rows, the experts' side tokens*choices rows, of which those that no
 * slot has are neither read nor written.  A value of rows[] outside
 * [0, tokens*choices) is a dropped slot; a row that two slots name is the
 * caller's mistake (which one is written is not defined).  With r = rows[t*choices + j]:
 *   sgemm_expert_dispatch       Y[r] = X[t]
 *   sgemm_expert_dispatch_int8  Q[r], scale[r] = row t of X as by sgemm_quantize_rows
 *   sgemm_expert_dispatch_grad  dX[t] = sum over j of dY[r]           (dispatch's gradient)
 *   sgemm_expert_combine        out[t] = sum over j of weights[t*choices + j] * Y[r]
 *   sgemm_expert_combine_grad   dY[r] = weights[t*choices + j] * dout[t],
 *                               dweights[t*choices + j] = sum over p of dout[t][p] * Y[r][p]
 * Sums run over the slots that are kept, in FP32 and in a fixed order (a token
 * with none gets zeros, a dropped slot's dweights is 0), and are rounded to
 * `type` once; weights and dweights are FP32.
 *
 * Checks, in order: handle, device, SGEMM_ERR_INVALID_VALUE (a negative size,
 * choices < 1, too many slots or experts, width above 2^30, an unknown type, a
 * leading dimension below max(1, width)), nothing is done when there is nothing to write,
 * SGEMM_ERR_NULL, SGEMM_ERR_INVALID_VALUE (a pointer not aligned to its element
 * size), SGEMM_ERR_ALIAS (an output overlaps an input or another output).  All
 * enqueue on `stream`, allocate nothing and do not synchronize. */
int sgemm_expert_sort(sgemm_handle_t h, int tokens, int choices, int experts, const int *ids, int *offsets,
                      int *rows, int *source, void *stream);
int sgemm_expert_dispatch(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *X, int ldx,
                          const int *rows, void *Y, int ldy, void *stream);
int sgemm_expert_dispatch_int8(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *X, int ldx,
                               const int *rows, int8_t *Q, int ldq, float *scale, void *stream);
int sgemm_expert_dispatch_grad(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *dY,
                               int lddy, const int *rows, void *dX, int lddx, void *stream);
int sgemm_expert_combine(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *Y, int ldy,
                         const int *rows, const float *weights, void *out, int ldo, void *stream);
int sgemm_expert_combine_grad(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *dout,
                              int lddo, const void *Y, int ldy, const int *rows, const float *weights, void *dY,
                              int lddy, float *dweights, void *stream);

/* A whole mixture-of-experts layer for a few tokens, in two launches:
 *
 *     out[t] = sum_j weights[t*choices + j] * D_e act(U_e X[t]),   e = ids[t*choices + j]
 *
 * with U_e = up_scale[e][f] * up[e][f][.] (rows x width, rows = hidden, with `gated`
 * 2 * hidden) and D_e = down_scale[e][d] * down[e][d][.] (width x hidden) in int8,
 * contiguous, as sgemm_run_int8_experts takes them (transB = 1).  act is silu(y) = y / (1 +
 * exp(-y)), with `gated` silu(y[f]) * y[hidden + f].  Choices whose id is outside
 * [0, experts) are left out, a token with none gets zeros; an expert that a token
 * names twice counts with both weights.
 *
 * X is taken as it is (16 or 32 bits) and the products are summed in FP32; the hidden
 * values keep 16 bits of fraction (24 with FP32 rows).  Elements (FP32) and hidden values of 3.396e38 and
 * more in magnitude, which BF16 rounds to infinity, count as infinities.  Only the experts that some
 * token names are read.
 *
 * The weights stream fastest where up and down are 16-byte aligned, width and hidden multiples of
 * 16, X 32-byte aligned and its rows multiples of 32 bytes apart.  Otherwise up to 3 bytes
 * beside X, up and down that share an aligned 4-byte word with theirs may be read, and do not
 * matter.  The chain of calls (sort, dispatch to 8 bits, two products, combine), which rounds tokens
 * and hidden values to 8 bits, takes less time from some 10 to 40 tokens on, sooner with
 * large experts.
 *
 * tokens up to 64, tokens * choices up to 1024, experts up to 1024, and the hidden values (4
 * bytes each, 6 with FP32 rows, hidden rounded up to 128, one row a choice) up to 48 MiB, else
 * SGEMM_ERR_INVALID_VALUE.  Other checks as for the routing calls. */
int sgemm_expert_layer_int8(sgemm_handle_t h, int type, int gated, int tokens, int choices, int experts, int width,
                            int hidden, const void *X, int ldx, const int *ids, const float *weights,
                            const int8_t *up, const float *up_scale, const int8_t *down, const float *down_scale,
                            void *out, int ldo, void *stream);

/* C <- alpha*A*B + beta*C with A, B, C in HOST memory, transfers overlapped
 * with compute.  dA, dB, dC are caller-owned DEVICE buffers of the same
 * shapes and leading dimensions (M*lda, K*ldb, M*ldc floats at least).  On a
 * handle-owned copy stream the library copies the first row panel of A (and
 * of C when beta != 0), then B in up to 8 column chunks, then the other row
 * panels; on `stream` it runs each piece of the GEMM (the same kernels and
 * rules as sgemm_run) as soon as its operands have landed -- the first row
 * panel in column blocks as B's chunks arrive, the middle panels as one
 * GEMM (two from four middle panels on, each started once its own panels
 * have landed), the last panel in column blocks; each segment's A rows may first be
 * copied transposed into the handle's re-layout workspace, once for all of
 * the segment's GEMMs -- and on a second copy stream it copies each finished
 * piece back to C while the rest computes.  Returns after enqueueing; C is complete when `stream`
 * reaches the point of the call (e.g. after cudaStreamSynchronize(stream)).
 * Page-locked host buffers give asynchronous copies; pageable ones work but
 * serialise.  The host and device windows must not be touched until then.
 * Same argument checks as sgemm_run (on the device pointers; SGEMM_ERR_NULL
 * also if a host pointer that is read or written is NULL), made before
 * anything is enqueued.  A CUDA error while enqueueing (after the checks)
 * returns SGEMM_ERR_CUDA with part of the copies and GEMMs possibly already
 * enqueued; synchronize `stream` before reusing the buffers.  The handle's
 * copy streams and events serve one call at a time: calls of the same handle
 * from several host threads must be serialised.  No allocation. */
int sgemm_run_host(sgemm_handle_t h, int M, int N, int K, float alpha,
                   const float *A, int lda, const float *B, int ldb,
                   float beta, float *C, int ldc,
                   float *dA, float *dB, float *dC, void *stream);

/* Host-only validation with exactly the rules sgemm_run applies (no CUDA call,
 * no handle): SGEMM_ERR_INVALID_VALUE if M, N or K < 0, lda < max(1, K),
 * ldb < max(1, N) or ldc < max(1, N); then, unless M == 0 or N == 0,
 * SGEMM_ERR_NULL if C is NULL, or if A or B is NULL while alpha != 0 and
 * K > 0; then SGEMM_ERR_ALIAS if the byte range of C's window overlaps that
 * of A's or B's window (only when A, B are read). */
int sgemm_check_args(int M, int N, int K, float alpha, const float *A, int lda,
                     const float *B, int ldb, float beta, const float *C, int ldc);

/* Synchronize the handle's device, then destroy it and free its device
 * memory.  SGEMM_ERR_BAD_HANDLE for NULL or an already destroyed handle. */
int sgemm_destroy(sgemm_handle_t h);

/* Pin a kernel variant for later calls of this handle (SGEMM_VARIANT_AUTO to
 * let the library choose).  SGEMM_ERR_INVALID_VALUE for an unknown value or
 * SGEMM_VARIANT_SCALE, which is chosen only by the alpha == 0 / K == 0 rule.
 * A pinned TMA variant fixes the tile; the re-layout mode still decides
 * whether operands are transposed first.  The 16-bit-input, int8 and 4-bit variants
 * act as SGEMM_VARIANT_AUTO for FP32 calls. */
int sgemm_set_variant(sgemm_handle_t h, int variant);

/* Set the handle's math mode (an sgemm_math_mode_t) for SGEMM_VARIANT_AUTO.
 * SGEMM_ERR_INVALID_VALUE for an unknown mode. */
int sgemm_set_math_mode(sgemm_handle_t h, int mode);

/* Set the handle's operand re-layout mode (an sgemm_relayout_t).
 * SGEMM_ERR_INVALID_VALUE for an unknown mode. */
int sgemm_set_relayout(sgemm_handle_t h, int mode);

/* Operands the handle's last successful sgemm_run / sgemm_run_ex copied
 * transposed before the GEMM: bit 0 A, bit 1 B (0 for none); -1 if `h` is
 * not a live handle. */
int sgemm_last_relayout(sgemm_handle_t h);

/* Size of the handle's re-layout workspace in floats (0 if it could not be
 * allocated, and then no operand is re-laid out); -1 if `h` is not a live
 * handle.  Transposed copies are stored with leading dimensions rounded up
 * to a multiple of 32 floats: A needs K * ceil32(M) floats per batch matrix,
 * B K * ceil32(N), both together the sum (the tensor-core variants' copies:
 * M * ceil32(K) for A, K * ceil32(N) for B). */
int64_t sgemm_relayout_capacity(sgemm_handle_t h);

/* The variant the handle's last successful sgemm_run enqueued (an
 * sgemm_variant_t), or -1 if there was none or `h` is not a live handle.
 * *splits (if non-NULL) receives the number of CTAs that share the K range of
 * a stream-K tile (rounded up; 1 when no tile was split). */
int sgemm_last_variant(sgemm_handle_t h, int *splits);

/* Number of kernel launches the handle's last successful call enqueued.
 * sgemm_run / sgemm_run_ex: 0 (nothing to do), one per transposed operand
 * (sgemm_last_relayout), then 1 to 3 for the GEMM: complete waves of whole
 * tiles; the stream-K CTAs of the last wave; and, for tiles larger than
 * 64 x 64, the kernel that adds the stream-K parts.  All on the same stream.
 * The 3xTF32 kernels: one launch per batch product after its copies.
 * -1 if `h` is not a live handle. */
int sgemm_last_launches(sgemm_handle_t h);

/* Wait for the handle's device to finish its work, then read and clear the
 * handle's device-side status word.  Returns SGEMM_OK, or
 * SGEMM_ERR_DEVICE_TIMEOUT if any kernel of the handle abandoned a bounded
 * wait, SGEMM_ERR_DEVICE_CHECK if a device-side index check failed (builds
 * with -DSGEMM_DEVICE_CHECKS; the check replaces the index with one in range,
 * so nothing is accessed out of bounds), or SGEMM_ERR_CUDA.  After a timeout the C of the calls since the last
 * check is undefined: some tiles may be unwritten and some may hold partial
 * sums or stale workspace contents.  On a timeout or a failed check this
 * call also clears the handle's stream-K arrival counters (a CTA that gave up
 * leaves its tile's counter unreset), so later calls on the handle are
 * correct again. */
int sgemm_get_device_status(sgemm_handle_t h);

/* Test hook: the stream-K workspace capacity, in partial tiles, that later
 * calls of the handle pass to their kernels for the device-side index checks
 * (0: the workspace's real size).  The plan still uses the real size, so a
 * limit below what a call needs makes a build with -DSGEMM_DEVICE_CHECKS
 * report SGEMM_ERR_DEVICE_CHECK for it -- every access stays inside the real
 * workspace -- and changes nothing in a build without the checks. */
int sgemm_debug_set_workspace_limit(sgemm_handle_t h, int tiles);

/* Test hook: put the handle in the state that a stream-K kernel which gave
 * up a bounded wait can leave behind -- every arrival counter nonzero and
 * the timeout bit set in the status word -- without running any kernel.
 * sgemm_get_device_status must then report the timeout and restore the
 * counters.  Synchronizes the device. */
int sgemm_debug_leave_aborted_state(sgemm_handle_t h);

/* Test hook: enqueue one small kernel that waits on a barrier nothing will
 * complete, gives up after `limit_ns` nanoseconds (clamped to [1e3, 1e9]),
 * records SGEMM_ERR_DEVICE_TIMEOUT in the handle's status word and returns.
 * It exercises the timeout path without faulting or hanging the GPU. */
int sgemm_debug_timeout_probe(sgemm_handle_t h, long long limit_ns, void *stream);

/* Measurement probe: enqueue `ctas` CTAs (0 = 4 per SM) of 256 threads, each
 * thread running 16 independent chains of packed FP32x2 FMAs for 8*iters
 * steps in registers (no memory traffic) and writing one sum to
 * sink[thread] (device memory of ctas*256 floats, caller-owned), and set
 * *flops (if non-NULL) to the FLOP the launch performs.  Timed with events
 * it gives the FP32 FMA rate the GEMM main loop is compared with.
 * SGEMM_ERR_NULL for a NULL sink; SGEMM_ERR_INVALID_VALUE if ctas < 0 or
 * iters < 1. */
int sgemm_debug_fma_probe(sgemm_handle_t h, int ctas, int iters, float *sink, long long *flops, void *stream);

/* Measurement probe of the TF32 tensor pipe: enqueue `clusters` clusters of
 * two CTAs (0 = one per pair of SMs; at most SMs/2), each issuing `iters`
 * K = 32 steps of the 3xTF32 CTA-pair kernel's MMA (tcgen05.mma
 * cta_group::2 kind::tf32, M = 256, N = 256, four K = 8 MMAs a step) on
 * operand tiles resident in shared memory, with no global-memory traffic,
 * and set *flops (if non-NULL) to the TF32 FLOP the launch performs.  Timed
 * with events it gives the measured TF32 rate; the 3xTF32 path spends three
 * TF32 MMAs per FP32 product, so its roofline is a third of it.  A wait that
 * runs out (bounded) is recorded in the handle's status word.
 * SGEMM_ERR_INVALID_VALUE if clusters < 0 or > SMs/2, or iters outside
 * 1 .. 2^20; SGEMM_ERR_WRONG_DEVICE off the handle's device. */
int sgemm_debug_tf32_probe(sgemm_handle_t h, int clusters, int iters, long long *flops, void *stream);

/* Measurement probe: `ctas` one-warp CTAs (0 = one per SM) each fill a 32 x 32
 * FP32 tile in shared memory with 0.001*(32*row + column) and read it
 * column-wise (lane l reads row l, k = 0..31) `iters` times -- the
 * transposed-operand access of page m.lqnn.cn/news/94381, section 4.2 -- with
 * a row stride of 32 floats (padded = 0: all 32 lanes in one bank, a 32-way
 * conflict per load) or 33 (padded = 1, the page's padding: 32 distinct
 * banks); lane l of CTA c writes its sum to sink[32*c + l] (ctas*32 floats,
 * caller-owned).  A control for the profiler's bank-conflict counters. */
int sgemm_debug_bank_probe(sgemm_handle_t h, int padded, int ctas, int iters, float *sink, void *stream);

/* Test hook: when `bytes` > 0, later launches of the handle's TMA variants
 * request `bytes` of dynamic shared memory instead of their own size, so a
 * value above the device limit makes the launch fail on the host
 * (SGEMM_ERR_LAUNCH) before anything runs.  0 restores normal launches. */
int sgemm_debug_set_smem_override(sgemm_handle_t h, int bytes);

/* How a call adds the partial sums of a tile whose K range is split over
 * stream-K CTAs (sgemm_debug_set_stream_k_sums).  Every mode adds a tile's
 * parts in ascending k order, so a tile split the same way gets the same
 * bits in every mode. */
typedef enum {
    SGEMM_SK_SUMS_AUTO = 0,     /* the library's choice (default) */
    SGEMM_SK_SUMS_LAST = 1,     /* the last CTA of the tile to arrive adds them all; the larger tiles
                                   split from 1.25 stream-K CTAs per tile as the 64 x 64 tile does */
    SGEMM_SK_SUMS_DEFERRED = 2, /* tiles larger than 64 x 64: every part stays in the workspace and a
                                   second kernel adds them (64 x 64 tiles: as LAST) */
    SGEMM_SK_SUMS_SHARED = 3    /* the CTAs whose K range ends in the tile wait for all its parts and
                                   add one slice of its elements each (every tile size) */
} sgemm_sk_sums_t;

/* Test hook: how later calls of the handle add the partial sums of a tile
 * whose K range is split over stream-K CTAs (sgemm_sk_sums_t).  Automatic:
 * for the tiles larger than 64 x 64, whichever of a second kernel and the
 * shared sums the library's time estimate prefers (and stream-K only where
 * it beats whole tiles); for the 64 x 64 tiles, whichever of the last CTA of
 * the tile to arrive and the shared sums it prefers (the last CTA reads the
 * parts one after another, which costs with many parts a tile).  The other
 * modes take the stream-K tail whenever a wave
 * has CTAs to spare (LAST: 1.25 per tile), so that every mode splits a call
 * the same way.  SGEMM_ERR_INVALID_VALUE for another value. */
int sgemm_debug_set_stream_k_sums(sgemm_handle_t h, int mode);

/* Test hook: cluster split-K CTAs per tile for later calls of the handle on
 * the whole-tile SIMT variants.  In cluster split-K, the `ksplit` CTAs of one
 * output tile form a thread-block cluster; CTA r takes K steps
 * [r*kt/ksplit, (r+1)*kt/ksplit) of the tile's kt steps of 32, the partial
 * tiles meet in distributed shared memory and each CTA adds a 1/ksplit slice
 * of them in ascending k order and writes it to C (one launch, no workspace).
 * 0 (the default): the library's choice, taken when all tiles x ksplit CTAs
 * fit in one wave and its time estimate beats whole tiles and stream-K.
 * 1: never.  2..8: that many CTAs per tile whenever K has at least as many
 * steps.  A tile split into ksplit parts this way gets the bits of the same
 * split through stream-K (ksplit * tiles stream-K CTAs).
 * SGEMM_ERR_INVALID_VALUE outside 0..8. */
int sgemm_debug_set_cluster_split(sgemm_handle_t h, int ksplit);

/* Test hook: the token tile of later int8 products on the tensor cores
 * (SGEMM_VARIANT_TC_I8) and the CTAs that share a tile's K range.  0, 0 (the default):
 * the library's choice.  tokens 16, 32 or 64 with ksplit 1, 2, 4 or 8 (taken down to
 * the 128-wide steps that K has), or tokens 128 or 256 (CTA pairs) with ksplit 1.  Every
 * one of them gives the same bits.  SGEMM_ERR_INVALID_VALUE otherwise. */
int sgemm_debug_set_int8_tile(sgemm_handle_t h, int tokens, int ksplit);

/* Test hook: the same for sgemm_run_fp4 on the tensor cores.  tokens 16, 32, 64 (taken up
 * to the call's tokens: such a tile is the only one) or 128 with ksplit 1, 2, 4 or 8 (taken
 * down to the 256-wide steps that K has), or 256 (CTA pairs) with ksplit 1; 0, 0: the
 * library's choice.  SGEMM_ERR_INVALID_VALUE otherwise. */
int sgemm_debug_set_fp4_tile(sgemm_handle_t h, int tokens, int ksplit);

/* Test hook: the number of stream-K CTAs of later calls' stream-K plans (the
 * last wave of the whole-tile variants, and the 64 x 64 split variant); 0 (the
 * default): the library's choice.  The count is kept within what a plan
 * allows -- more CTAs than the tail has tiles (the split variant: at least
 * two per tile), at most a wave of them and the workspace's partial tiles --
 * and a call whose plan has no stream-K part is unaffected.
 * SGEMM_ERR_INVALID_VALUE for a negative count. */
int sgemm_debug_set_stream_k_ctas(sgemm_handle_t h, int ctas);

/* Test hook: how the stream-K CTAs of later calls of the handle share the K
 * steps of the tiles they split.  The K steps lie on a line, 16 positions
 * each, with `gap` positions of no work before every tile but the first; CTA
 * q of G takes the K steps whose last position falls in its equal share
 * [gap + floor(q*V/G), gap + floor((q+1)*V/G)) of the V positions.  A CTA whose
 * range runs into a further tile stores one more partial tile, and the gap
 * charges it for that with fewer K steps.  gap = 0 is the even split
 * (floor(q*T/G) .. floor((q+1)*T/G) of the T K steps).  -1 (the default): the
 * library's choice among 0, 4, .., 24, the one whose busiest CTA has the least
 * work by its estimate; 0..128: that charge, where every CTA then gets at
 * least one and at most a tile's K steps (else 0).  Any charge gives a valid
 * split whose tiles' parts are added in ascending k order; splits differ in
 * where a tile's K range is cut, so results of different charges may differ
 * in the last bits.  SGEMM_ERR_INVALID_VALUE outside -1..128. */
int sgemm_debug_set_stream_k_gap(sgemm_handle_t h, int gap);

/* Test hook: the plan sgemm_run_ex would follow for a call, computed on the
 * host with no handle, no device and no CUDA call, from the device facts a
 * handle records (`num_sms`; `ctas_per_sm`, SGEMM_VARIANT_COUNT_ entries
 * indexed by sgemm_variant_t: resident CTAs per SM of each TMA variant) and
 * its settings (re-layout workspace size in floats, re-layout mode, math
 * mode, pinned variant).  `aligned` says which operands the TMA can read as
 * stored: bit 0 A, bit 1 B, each set when the operand is 16-byte aligned with
 * its leading dimension (and batch stride) a multiple of 4 (3: both, as for
 * any call on 16-byte aligned buffers with such leading dimensions).  An
 * operand it cannot read is copied transposed into the re-layout workspace
 * when the mode allows and the copy fits and pays; else the call runs on the
 * generic kernel.  out[0..12] receives: the
 * kind (0 nothing to do, 1 the beta*C quick path, 2 tensor-core kernel, 3
 * generic kernel, 4 TMA SIMT kernel), the variant that runs, the operands
 * copied transposed first (bit 0 A, bit 1 B), the TMA operand layout (0 NN,
 * 1 TN, 2 NT), the whole tiles run in complete waves, the stream-K CTAs, the
 * tiles of the call, the kernel launches, the CTAs per stream-K tile, and how
 * the stream-K tiles' parts are added (0 by the last CTA of each tile to
 * arrive, or without stream-K; 1 by a second kernel; 2 shared by the CTAs
 * whose K range ends in the tile), the cluster split-K CTAs per tile (1:
 * none), 1 when the 3xTF32 pair kernel reads B stored N x K (an operand
 * stored K x N is then copied transposed first; 0: B stored K x N), and the
 * stream-K split's boundary charge (sgemm_debug_set_stream_k_gap; 0: the
 * even split, or no stream-K).
 * SGEMM_ERR_NULL for a NULL array, SGEMM_ERR_INVALID_VALUE for an argument out
 * of range. */
int sgemm_debug_plan(int num_sms, const int *ctas_per_sm, long long relayout_floats, int relayout_mode,
                     int math_mode, int pinned, int transA, int transB, int M, int N, int K, float alpha,
                     int batch, long long strideA, long long strideB, int aligned, int *out);

/* C <- alpha*A*B + beta*C without allocating anything, for callers that cannot
 * allocate GPU memory (allocator implementations that must not re-enter the
 * allocator, frameworks whose allocator has reserved the device memory, hosts
 * that forbid device allocation after start-up).  The pages have no
 * counterpart: this is a deployment convenience, not part of the method.
 *
 * Same arguments, rules and results as sgemm_run, but no handle: it runs the
 * 64 x 64 stream-K kernel with its partial tiles, tile counters and status word
 * in a fixed scratch array compiled into the library (8 MiB + 4 KiB + 256 B,
 * held on every GPU that loads the library until the process exits).
 * Limit: at most 512 output tiles of 64 x 64, i.e. ceil(M/64)*ceil(N/64) <= 512;
 * larger problems return SGEMM_ERR_SCRATCH_TOO_SMALL and enqueue nothing.
 * alpha == 0 or K == 0, and operands TMA cannot describe, take the same
 * scratch-free kernels as sgemm_run.  It calls no cudaMalloc or cudaFree.
 * All calls share the scratch and it keeps the last call's contents: each call
 * clears the counters and status word it uses on `stream` first, and calls that
 * overlap on the GPU (unordered streams) race and give wrong results.  The
 * first call on a device, with that device current, looks up the scratch's
 * device address and sets the kernel up; make that first call before any
 * stream capture, and do not reset the device (cudaDeviceReset) between
 * calls: the address found is kept for the life of the process.  A
 * device-side timeout leaves the tiles it hit unwritten and cannot be
 * reported by this entry point. */
int sgemm_run_noalloc(int M, int N, int K, float alpha, const float *A, int lda,
                      const float *B, int ldb, float beta, float *C, int ldc, void *stream);

/* Human-readable name of a status value (never NULL). */
const char *sgemm_status_string(int status);

/* Human-readable name of a variant value (never NULL). */
const char *sgemm_variant_name(int variant);

/* Library version, major*10000 + minor*100 + patch. */
int sgemm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_H */
