/*
 * libgemm — tiled mixed-precision matrix multiply-accumulate D = A x B + C
 * on AMD Instinct MI355X (gfx950), as hand-written HIP kernels behind a C ABI.
 *
 * The operation (sources, by page title and section):
 *  - D = A*B + C, fused multiply-accumulate with low-precision A, B and a
 *    high-precision accumulator; D has the precision of C:
 *    "深入CUDA Tensor Core与WMMA：从基础原理到高性能混合精度矩阵乘实战",
 *    section 2.2 "核心运算：融合矩阵乘累加（MMA）".
 *  - Element definition C[i,j] = sum over k in [0,K) of A[i,k]*B[k,j]:
 *    "矩阵乘法优化可视化学习文档", section 1 "先建立心智模型".
 *  - Row-major / column-major storage with a leading dimension (stride, in
 *    elements, between consecutive rows resp. columns): "深入CUDA Tensor Core
 *    与WMMA…", sections 3.2 (2x3 example) and 4.2 (ldm); "CUDA算子优化(5)：
 *    WMMA矩阵乘法", section "WMMA API解释" items (2) and (3).
 *  - In-place C = A*B + C, and satf (saturate to finite): +Inf -> +MAX_NORM,
 *    -Inf -> -MAX_NORM, NaN -> +0: "CUDA算子优化(5)：WMMA矩阵乘法",
 *    section "WMMA API解释" item (5) mma_sync.
 *  - fp16-accumulate HGEMM variant (fp16 A, B, C, D):
 *    "hgemm_mma_m16n8k16_naive_kernel", section 1.1 "m16n8k16 指令规格".
 *  - 8-bit float inputs (fp8): the per-architecture precision lists of
 *    "深入CUDA Tensor Core与WMMA…", section 2.3; here the OCP E4M3 and E5M2
 *    formats gfx950's matrix cores take.
 *  - int8 inputs with an int32 accumulator: the fragment type lists of
 *    "CUDA算子优化(5)：WMMA矩阵乘法" (char operands, int accumulator) and
 *    "深入CUDA Tensor Core与WMMA…", section 2.3 (INT8 on the matrix units).
 *
 * Readings where the pages leave a step open:
 *  - C and D are row-major (C(i,j) = C[i*ldc + j]); C has the output dtype.
 *  - acc_dtype GEMM_F16 selects the HGEMM variant: C, D and MAX_NORM are fp16.
 *    The sum itself is accumulated in fp32 (gfx950's f16 MFMAs accumulate in
 *    fp32) and rounded once to fp16, the accuracy the page on mixed precision
 *    asks for (section 7.1 "常见坑点", item 5).
 *  - satf is applied once, to the value rounded to out_dtype; MAX_NORM is the
 *    largest finite value of out_dtype.
 *  - Rounding to fp16 / bf16 is round-to-nearest-even.
 *  - Nothing outside rows [0,M) and columns [0,N) of D is written.  A and B
 *    are read in aligned 16-byte blocks (vector path) or element by element
 *    (other alignments): every block read holds at least one element of the
 *    M x K resp. K x N matrix, so bytes of the leading-dimension padding next
 *    to those elements (and up to 15 bytes past the last element) may be
 *    read, but never affect D; nothing else outside the matrices is read.
 *  - int8 (in_dtype GEMM_I8, acc and out GEMM_I32): the sum is exact; the
 *    result (+ C) wraps modulo 2^32, or with satf is clamped to the int32
 *    range.  satf needs K < 2^17, where the int32 accumulator cannot wrap.
 */
#ifndef LIBGEMM_H
#define LIBGEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Storage order of A and B. */
typedef enum {
    GEMM_ROW_MAJOR = 0, /* X(r,c) = X[r*ld + c] */
    GEMM_COL_MAJOR = 1  /* X(r,c) = X[c*ld + r] */
} gemm_layout_t;

/* Element types. */
typedef enum {
    GEMM_F32 = 0,  /* IEEE binary32 */
    GEMM_F16 = 1,  /* IEEE binary16 */
    GEMM_BF16 = 2, /* bfloat16 (upper half of binary32) */
    GEMM_I8 = 3,   /* two's-complement 8-bit integer (A, B)  */
    GEMM_I32 = 4,  /* two's-complement 32-bit integer (C, D, accumulator) */
    GEMM_FP8_E4M3 = 5, /* OCP 8-bit float E4M3 (A, B): bias 7, max 448, NaN, no Inf */
    GEMM_FP8_E5M2 = 6  /* OCP 8-bit float E5M2 (A, B): bias 15, IEEE-style Inf/NaN */
} gemm_dtype_t;

/* Return codes.  GEMM_OK means "validated and enqueued". */
typedef enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_DIM = -1,    /* M, N or K negative, or above 2^31-1        */
    GEMM_ERR_INVALID_LD = -2,     /* a leading dimension shorter than its matrix */
    GEMM_ERR_NULL_PTR = -3,       /* NULL A, B or D for a non-empty operation    */
    GEMM_ERR_UNSUPPORTED = -4,    /* dtype combination not provided              */
    GEMM_ERR_INVALID_LAYOUT = -5, /* layout not GEMM_ROW_MAJOR / GEMM_COL_MAJOR  */
    GEMM_ERR_ALIASING = -6,       /* D overlaps A or B, or C partially overlaps D */
    GEMM_ERR_HIP = -7,            /* the HIP runtime reported an error           */
    GEMM_ERR_INVALID_CONFIG = -8, /* gemm_run_config: no such config, or the
                                     config cannot run this problem            */
    GEMM_ERR_SCRATCH_TOO_SMALL = -9 /* gemm_run_noalloc: the split-K partial
                                     sums need more than its fixed scratch;
                                     a call with a workspace of the caller's:
                                     workspace_bytes too small                */
} gemm_status_t;

/*
 * D = A x B + C on the device.
 *
 *   M, N, K      problem size: A is M x K, B is K x N, C and D are M x N.
 *                M == 0 or N == 0: nothing to do, returns GEMM_OK.
 *                K == 0: D = satf(round(C)) (or +0 when C is NULL).
 *   A, lda, layoutA   device pointer to in_dtype elements; lda >= K when
 *                row-major, >= M when col-major (and >= 1).
 *   B, ldb, layoutB   device pointer to in_dtype elements; ldb >= N when
 *                row-major, >= K when col-major (and >= 1).
 *   C, ldc       device pointer to out_dtype elements, row-major, ldc >= N;
 *                may be NULL (C = 0).  C == D with ldc == ldd is the in-place
 *                update C = A x B + C; any other overlap of C and D is rejected.
 *   D, ldd       device pointer to out_dtype elements, row-major, ldd >= N.
 *   in_dtype     GEMM_F16, GEMM_BF16, GEMM_FP8_E4M3, GEMM_FP8_E5M2 (A and B
 *                both of that type), or GEMM_I8 (A and B int8).
 *   acc_dtype    GEMM_F32 (out_dtype F32, F16 or BF16; any float input), or GEMM_F16 with
 *                in_dtype == out_dtype == GEMM_F16 (HGEMM), or GEMM_I32 with
 *                in_dtype GEMM_I8 and out_dtype GEMM_I32.
 *   out_dtype    dtype of C and D.
 *   satf         nonzero: +Inf -> +MAX_NORM, -Inf -> -MAX_NORM, NaN -> +0;
 *                for int32 output: clamp to [-2^31, 2^31-1] instead of wrapping
 *                (int8 with K >= 2^17 and satf: GEMM_ERR_UNSUPPORTED).
 *   stream       a hipStream_t (NULL = the null stream).  The work is enqueued
 *                on it; the call does not wait for it.
 *
 * Ownership: every pointer is owned by the caller and must stay valid until
 * the stream reaches the enqueued work.  Problems split along K (M <= 16),
 * and large calls (M*N*K >= 2^30) whose A or B misses the vector loads only
 * by alignment (that operand is first copied there with 16-byte lines), use
 * a device workspace the library owns: one per (device, stream) pair,
 * allocated with hipMalloc on first need and grown on demand.  A call holds
 * the workspace's lock from taking the buffer until all of its launches are
 * enqueued, so calls from several host threads on one stream are enqueued
 * one after the other; an outgrown buffer is never freed (work enqueued
 * earlier may still use it).  Workspaces are kept until the process exits.
 *
 * Errors: argument errors are detected on the host before anything is
 * enqueued, and nothing is written.  GEMM_ERR_HIP reports a launch or
 * allocation failure (the launch's own status, not an earlier error); D is
 * then not written, except that a call whose later launch fails has already
 * enqueued the earlier ones (an operand copy, a split-K slice kernel), which
 * write only the workspace.
 * Faults inside the kernels surface at the next synchronisation of the
 * stream.
 *
 * Speed: vector loads are used where A and B base pointers are 16-byte
 * aligned and lda, ldb are multiples of 16 bytes (the pages' ldm rule), in
 * every layout (operands contiguous along M or N are transposed on the way
 * to LDS); large calls with other operands copy them into the workspace
 * with 16-byte lines first (see Ownership), and the rest run correct
 * element-wise loads.  C and D
 * are read and written four elements at a time where their base pointers
 * are aligned to four elements, ldc and ldd are multiples of 4 and C is
 * row-major (and, for gemm_run_ex, a per-column bias is 16-byte aligned);
 * otherwise element by element.
 *
 * fp8 accuracy: gfx950's fp8 MFMA adds the products of each output in
 * groups of 8 consecutive k, aligned to the largest product of the group:
 * what lies below 2^-13 of that product is lost (measured, E4M3 and E5M2),
 * before the fp32 accumulation.  Each product is then off by less than
 * 2^-13 * max|a| * max|b|.  Products of inputs of similar magnitude, and
 * integer-valued inputs, come out exact.
 */
int gemm_run(int64_t M, int64_t N, int64_t K,
             const void *A, int64_t lda, int layoutA,
             const void *B, int64_t ldb, int layoutB,
             const void *C, int64_t ldc,
             void *D, int64_t ldd,
             int in_dtype, int acc_dtype, int out_dtype,
             int satf, void *stream);

/*
 * gemm_run without any device allocation, for callers that cannot allocate:
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, validation and results as gemm_run (the same
 * kernels, bit-identical D), except for large calls whose operands gemm_run
 * would copy into its workspace for alignment: this call runs those with
 * element-wise loads instead (the same results to the stated tolerances;
 * slower).  Where gemm_run would take its split-K partial
 * sums from a workspace it allocates (M <= 16), this call uses a scratch
 * array of fixed size compiled into the library: 32 MiB of device memory per
 * GPU the library runs on, held until the process ends.  Problems whose
 * partial sums (splits * M * N * 4 bytes) exceed it return
 * GEMM_ERR_SCRATCH_TOO_SMALL before anything is enqueued (on a 256-CU
 * MI355X no problem needs more than about 17 MB).  Every call on a
 * GPU shares that GPU's scratch, and nothing guards it: calls that can
 * overlap on one GPU (other streams, other host threads) race on it and must
 * be ordered by the caller.  The scratch needs no clearing (each call writes
 * every partial sum it reads).  The call makes no hipMalloc, hipFree or other
 * allocating call; its first call on a device looks up the scratch's device
 * address (hipGetSymbolAddress), which allocates no memory of its own: the
 * scratch is part of the library's device code object.  The call enqueues
 * only kernel launches (no memset or copy nodes), so it can be captured into
 * a HIP graph once the device is initialised; a replay computes what the
 * captured call would (tested: replays between eager calls of both entry
 * points, bit-identical to the eager result).
 */
int gemm_run_noalloc(int64_t M, int64_t N, int64_t K,
                     const void *A, int64_t lda, int layoutA,
                     const void *B, int64_t ldb, int layoutB,
                     const void *C, int64_t ldc,
                     void *D, int64_t ldd,
                     int in_dtype, int acc_dtype, int out_dtype,
                     int satf, void *stream);

/* Static text for a gemm_status_t value ("unknown status" otherwise). */
const char *gemm_status_string(int status);

/*
 * The tile-shape table.  Each entry is one tiling (block tile, wave grid,
 * MFMA shape, split-K policy); the dispatcher of gemm_run picks an entry per
 * shape class.  Tiling and autotuning by shape: "矩阵乘法优化可视化学习文档",
 * section 6 "常用优化方法总表" (Tiling, Autotuning rows).
 *
 * gemm_num_configs: number of entries.
 * gemm_config_name: static text naming entry `config_id` (NULL if out of range).
 * gemm_select_config: the entry gemm_run would use for this problem with
 *                16-byte aligned operand lines, or a negative gemm_status_t
 *                if the arguments are invalid.  Entries whose kernels load
 *                operands straight into LDS ("large_dma...", and the 8-bit
 *                "i8_large_dma..." and "fp8_large_dma8...") accept only
 *                16-byte aligned operand lines, and "i8_large_dma_..." (the
 *                four-wave 16x16x64 one) only K-contiguous operands (A
 *                row-major and B column-major as the kernels see them: a
 *                column-major D swaps and flips them): with other operands
 *                gemm_run runs the register-staged 256x256 entry of the
 *                input type instead, and gemm_run_config forced to such an
 *                entry returns GEMM_ERR_INVALID_CONFIG.
 */
int gemm_num_configs(void);
const char *gemm_config_name(int config_id);
int gemm_select_config(int64_t M, int64_t N, int64_t K, int layoutA, int layoutB,
                       int in_dtype, int acc_dtype, int out_dtype);

/*
 * gemm_run with the tile-table entry forced to `config_id` (same arguments,
 * same validation, same results up to summation order).  For tests and
 * benchmarks that must reach every entry.  GEMM_ERR_INVALID_CONFIG if the
 * entry does not exist.
 */
int gemm_run_config(int config_id,
                    int64_t M, int64_t N, int64_t K,
                    const void *A, int64_t lda, int layoutA,
                    const void *B, int64_t ldb, int layoutB,
                    const void *C, int64_t ldc,
                    void *D, int64_t ldd,
                    int in_dtype, int acc_dtype, int out_dtype,
                    int satf, void *stream);

/*
 * Host-only argument check of gemm_run (no HIP call, no device needed):
 * returns GEMM_OK or the error gemm_run would return before enqueuing, except
 * the int8 satf limit on K, which depends on satf.
 */
int gemm_validate(int64_t M, int64_t N, int64_t K,
                  const void *A, int64_t lda, int layoutA,
                  const void *B, int64_t ldb, int layoutB,
                  const void *C, int64_t ldc,
                  const void *D, int64_t ldd,
                  int in_dtype, int acc_dtype, int out_dtype);

/* ===================================================== extended epilogue
 *
 * D = act( alpha * (A x B) + beta * C + bias ), rounded once to out_dtype,
 * then satf; C and D each row- or column-major.
 *
 * Sources: "矩阵乘法优化可视化学习文档", section 6 "常用优化方法总表"
 * (Epilogue fusion row: bias, activation and scale applied before the
 * write-back) and section 8 (bias/activation fused at the final store, and
 * the check that the fused result matches the unfused reference); the
 * accumulator load/store layouts mem_row_major / mem_col_major of
 * "CUDA算子优化(5)：WMMA矩阵乘法", section "WMMA API解释" items (3) and (4).
 *
 * Readings (the pages name bias, activation and scale but fix none of them):
 *  - scale is the usual pair alpha (on the product) and beta (on C); with
 *    beta == 0, C is not read (it may hold anything, NaN included);
 *  - bias holds one fp32 value per column j of D, added after the scaling;
 *  - GEMM_ACT_RELU is max(x, 0) with NaN kept and -0 -> +0; GEMM_ACT_GELU is
 *    x * Phi(x) = x/2 * (1 + erf(x / sqrt 2)), with GELU(+Inf) = +Inf and
 *    GELU(-Inf) = 0;
 *  - everything between the product and the final rounding is fp32; GELU
 *    evaluates erfc by Abramowitz & Stegun formula 7.1.26 (absolute error
 *    <= 1.5e-7), i.e. GELU to within about 2.2e-7 * max(1, |x|).
 */
typedef enum {
    GEMM_ACT_NONE = 0,
    GEMM_ACT_RELU = 1,
    GEMM_ACT_GELU = 2,
    GEMM_ACT_SILU = 3  /* x / (1 + exp(-x)); gemm_moe_run, gemm_checkpoint_act_grad only */
} gemm_activation_t;

typedef struct {
    float alpha;          /* scale of A x B (1.0f: none)                       */
    float beta;           /* scale of C (1.0f: none; 0.0f: C is not read)      */
    const float *bias;    /* device pointer to N fp32 values, or NULL          */
    int activation;       /* gemm_activation_t                                 */
    int layoutC;          /* gemm_layout_t of C: row-major C(i,j) = C[i*ldc+j],
                             column-major C(i,j) = C[j*ldc+i]                  */
    int layoutD;          /* gemm_layout_t of D, same convention               */
} gemm_epilogue_t;

/*
 * gemm_run with the extended epilogue.  `epi` == NULL, or
 * {1, 1, NULL, GEMM_ACT_NONE, GEMM_ROW_MAJOR, GEMM_ROW_MAJOR}, is exactly
 * gemm_run (bit-identical results).  Other arguments as for gemm_run, except:
 *   ldc, ldd     >= N for a row-major matrix, >= M for a column-major one.
 *   C == D       (in place) needs ldc == ldd and layoutC == layoutD.
 *   bias         N fp32 values on the device; must not overlap D.
 * Errors, in addition to gemm_run's: an activation outside gemm_activation_t,
 * or int8 inputs with anything but the plain epilogue (alpha = 1, beta 1 or
 * 0, no bias, no activation; C/D layouts are fine) -> GEMM_ERR_UNSUPPORTED; layoutC / layoutD not a gemm_layout_t ->
 * GEMM_ERR_INVALID_LAYOUT; bias overlapping D, or C == D with different
 * layouts or leading dimensions -> GEMM_ERR_ALIASING.
 *
 * Speed: a column-major D runs the row-major kernels on D^T = B^T x A^T (the
 * operands swap roles, no data moves); C in the other layout than D, and
 * a bias pointer that is not 16-byte aligned, take the element-wise store
 * path of edge tiles.  With an fp32 D (leading dimensions of C and D
 * multiples of 4, 16-byte aligned C, D and bias) and K a multiple of the
 * tile's K step, the register-staged entries apply the whole epilogue
 * from registers; other calls stage each tile through LDS first.  GELU
 * costs about 20 vector instructions per output element.
 */
int gemm_run_ex(int64_t M, int64_t N, int64_t K,
                const void *A, int64_t lda, int layoutA,
                const void *B, int64_t ldb, int layoutB,
                const void *C, int64_t ldc,
                void *D, int64_t ldd,
                int in_dtype, int acc_dtype, int out_dtype,
                int satf, const gemm_epilogue_t *epi, void *stream);

/* gemm_run_ex with the tile-table entry forced (see gemm_run_config). */
int gemm_run_ex_config(int config_id,
                       int64_t M, int64_t N, int64_t K,
                       const void *A, int64_t lda, int layoutA,
                       const void *B, int64_t ldb, int layoutB,
                       const void *C, int64_t ldc,
                       void *D, int64_t ldd,
                       int in_dtype, int acc_dtype, int out_dtype,
                       int satf, const gemm_epilogue_t *epi, void *stream);

/* Host-only argument check of gemm_run_ex (see gemm_validate). */
int gemm_validate_ex(int64_t M, int64_t N, int64_t K,
                     const void *A, int64_t lda, int layoutA,
                     const void *B, int64_t ldb, int layoutB,
                     const void *C, int64_t ldc,
                     const void *D, int64_t ldd,
                     int in_dtype, int acc_dtype, int out_dtype,
                     const gemm_epilogue_t *epi);

/* ============================================== quantised linear layers
 *
 * An int8 product with a scale for each row of A (a token) and each column of
 * D (an output channel), and the operator that makes such an A from 16-bit or
 * 32-bit activations.  Both enqueue one kernel (gemm_run_scaled one for every
 * 4 GiB of A and of B and every 2^27 rows and columns, gemm_quantize_rows one for
 * every 2^21 rows), allocate nothing and use no workspace, so they can be captured
 * into a HIP graph, and calls on different streams do not touch each other.
 *
 * gemm_quantize_rows: for each row i of X (M x K, row-major, ldx >= K),
 *
 *   a = max_k |X(i,k)|,   scales[i] = a / 127,
 *   Q(i,k) = X(i,k) * 127 / a, rounded to nearest even,
 *
 * so Q lies in [-127, 127] and X(i,k) = scales[i] * Q(i,k) to within half a
 * step (scales[i] / 2).
 *   in_dtype     GEMM_F16, GEMM_BF16 or GEMM_F32 (X).
 *   Q, ldq       device pointer to int8 elements, row-major, ldq >= K.  Nothing
 *                outside rows [0,M) and columns [0,K) is written.
 *   scales       device pointer to M fp32 values.
 * A row of zeros (or K == 0) gets scale 0 and zeros.  A row that holds an Inf or
 * a NaN gets scale NaN and zeros, so that a product with it is NaN, not a
 * number that looks right.
 * Accuracy: Q is the correctly rounded value of the exact quotient (ties to
 * even) for every finite row; scales[i] is a / 127 rounded once to fp32.
 * Speed: 16-byte loads and stores where X and Q are 16-byte aligned with ldx
 * and ldq multiples of 16 bytes; element by element otherwise.
 * Errors: GEMM_ERR_INVALID_DIM, GEMM_ERR_INVALID_LD, GEMM_ERR_NULL_PTR (a
 * pointer that a non-empty operation needs), GEMM_ERR_UNSUPPORTED (in_dtype),
 * GEMM_ERR_ALIASING (X, Q and scales must not overlap), GEMM_ERR_HIP.
 */
int gemm_quantize_rows(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype, void *Q,
                       int64_t ldq, float *scales, void *stream);

/* Host-only argument check of gemm_quantize_rows (see gemm_validate). */
int gemm_validate_quantize_rows(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype,
                                const void *Q, int64_t ldq, const float *scales);

/*
 * gemm_run_scaled: D = act( alpha * (A x B)(i,j) * scaleA[i] * scaleB[j]
 *                           + beta * C(i,j) + bias[j] ),
 * A x B the exact int32 sum of int8 products, rounded once to out_dtype, then
 * satf.  Arguments as for gemm_run_ex, with
 *   in_dtype     GEMM_I8, acc_dtype GEMM_I32, out_dtype GEMM_F32, GEMM_F16 or
 *                GEMM_BF16 (C and D), K < 2^17 (the int32 sum cannot wrap).
 *   scaleA       device pointer to M fp32 values, one for each row of A, or
 *                NULL (1).
 *   scaleB       device pointer to N fp32 values, one for each column of B, or
 *                NULL (1).
 *   epi          gemm_epilogue_t (alpha, beta, bias, activation, layouts of C
 *                and D), or NULL.
 * Between the exact sum and the final rounding everything is fp32: the sum is
 * rounded to fp32, multiplied by the row's scale, the column's scale and alpha
 * in this order (three roundings, each 2^-24 relative), then beta * C and bias
 * are added.  Where K == 0 the product is 0, whatever the scales.
 * Errors as gemm_run_ex, and: another dtype combination, or K >= 2^17 ->
 * GEMM_ERR_UNSUPPORTED; D overlapping scaleA or scaleB -> GEMM_ERR_ALIASING.
 *
 * Speed: vector loads as for gemm_run.  With K-contiguous operands (row-major A,
 * column-major B) and vector loads, up to 32 rows stream B from memory once, a
 * column block for each workgroup, and calls of few output tiles take deeply
 * pipelined ones; other calls run the int8 tiles.  Nothing splits K between
 * workgroups, so few rows with a row-major B leave most of the GPU idle (1 to 128 x
 * 4096 x 16384: 102 us, with a column-major B 14 to 30).  Operands that miss the
 * vector loads are read element by element (gemm_run copies large ones into its
 * workspace first; this call has none): lines of 16392 instead of 16384 bytes take 1
 * x 4096 x 16384 from 14 to 684 us.  C is read element by element too (4096^3 in bf16:
 * 74 us, 117 with C).
 */
int gemm_run_scaled(int64_t M, int64_t N, int64_t K,
                    const void *A, int64_t lda, int layoutA,
                    const void *B, int64_t ldb, int layoutB,
                    const float *scaleA, const float *scaleB,
                    const void *C, int64_t ldc,
                    void *D, int64_t ldd,
                    int in_dtype, int acc_dtype, int out_dtype,
                    int satf, const gemm_epilogue_t *epi, void *stream);

/* Host-only argument check of gemm_run_scaled (see gemm_validate). */
int gemm_validate_scaled(int64_t M, int64_t N, int64_t K,
                         const void *A, int64_t lda, int layoutA,
                         const void *B, int64_t ldb, int layoutB,
                         const float *scaleA, const float *scaleB,
                         const void *C, int64_t ldc,
                         const void *D, int64_t ldd,
                         int in_dtype, int acc_dtype, int out_dtype,
                         const gemm_epilogue_t *epi);

/* ================================================ mixture of experts
 *
 * A whole mixture-of-experts layer for a few tokens (T <= 64: decoding), from
 * the router's logits to the layer's output, in two kernels.  For each token t
 * with logits l (the router's product, e.g. by gemm_run into fp32):
 *
 *   chosen   the topk experts of largest l, ties to the lower index
 *   w_e    = exp(l_e) / sum over all experts of exp(l), or with renormalize
 *            / sum over the chosen experts
 *   h_e    = act(x G_e^T) * (x U_e^T)         elementwise, I values
 *   y      = sum over the chosen e of w_e (h_e D_e^T)
 *
 * An expert at -Inf is not chosen, so a token may have fewer than topk experts;
 * one whose logits are all -Inf has y = 0.  A token with a NaN or +Inf among
 * its logits has y = NaN.  Experts that no token chose are not read.
 *
 * gemm_moe_t describes the layer:
 *   H, I, E, topk   model width, inner width, experts (<= 1024), experts of a
 *                token (<= 32, <= E); H, I in [1, 2^19]
 *   w_dtype      GEMM_F16 or GEMM_BF16 (then the type of x), or GEMM_I8
 *   W1, ld1      E x 2I rows of H elements, lines ld1 >= H elements apart: rows
 *                [0, I) of an expert are its gate G, rows [I, 2I) its up U
 *   W2, ld2      E x H rows of I elements, lines ld2 >= I elements apart: D
 *   scale1, scale2   GEMM_I8: one fp32 scale for each row of W1 (E x 2I) and W2
 *                (E x H), contiguous; the weight is scale * int8.  Else unused.
 *   activation   act: GEMM_ACT_SILU, GEMM_ACT_GELU or GEMM_ACT_RELU
 *   renormalize  nonzero: the chosen weights sum to 1
 *
 * gemm_moe_run:
 *   T            tokens, 0 to 64.  T == 0: nothing to do, returns GEMM_OK.
 *   X, ldx       T x H elements of in_dtype (GEMM_F16 or GEMM_BF16), row-major
 *   logits, ldl  T x E fp32, row-major
 *   D, ldd       T x H elements of in_dtype, row-major; nothing outside is written
 *   workspace    device memory of at least gemm_moe_workspace(T, layer) bytes,
 *                of any content, owned by the caller, written by the call.  A call
 *                must not overlap another one (or a graph's replay) that uses the
 *                same workspace, unless the caller orders them; calls with
 *                workspaces of their own may overlap freely.
 * The call enqueues two kernels and allocates nothing, so it can be captured
 * into a HIP graph; the routing is found on the device, and a replay follows the
 * logits of its own time.  The same call gives the same bits.
 *
 * Accuracy: products and sums are fp32, as are the softmax and everything
 * between, and y is rounded once at the end.  The second product takes h as the sum
 * of two values of in_dtype: 16 significant bits for bf16; for fp16 22, of h times a
 * power of two that follows the largest value of its row (one token and expert), so
 * that h may lie anywhere in fp32's range, and what is below 2^-34 of the row's
 * largest value is lost.  int8 weights are converted exactly and their scales
 * applied to the fp32 sums.  An Inf in a chosen expert's W2 gives NaN.
 *
 * Speed: bound by the chosen experts' weights, each read once.  16-byte loads
 * where X, W1 and W2 are all 16-byte aligned with lines of whole 16 bytes; element
 * by element, all three, otherwise (slow).  With more than 256 experts and fewer than
 * that many pairs of token and expert the routing outweighs them (8 tokens, top 8 of
 * int8 experts of 512 x 256: 48 us with 256 experts, 190 with 512, 1204 with 1024).
 *
 * Errors: GEMM_ERR_INVALID_DIM (T < 0; H, I, E or topk out of range above or
 * topk > E), GEMM_ERR_UNSUPPORTED (T > 64, E > 1024, topk > 32, a dtype or
 * activation not named above), GEMM_ERR_INVALID_LD (a line shorter than its
 * row, or longer than 2^24 elements), GEMM_ERR_NULL_PTR,
 * GEMM_ERR_ALIASING (D or the workspace overlapping another argument),
 * GEMM_ERR_SCRATCH_TOO_SMALL, GEMM_ERR_HIP (D is then not written).
 */
typedef struct {
    int64_t H, I, E, topk;
    const void *W1;
    int64_t ld1;
    const void *W2;
    int64_t ld2;
    const float *scale1, *scale2;
    int w_dtype;
    int activation;
    int renormalize;
} gemm_moe_t;

int gemm_moe_run(int64_t T, const gemm_moe_t *layer, const void *X, int64_t ldx,
                 const float *logits, int64_t ldl, void *D, int64_t ldd, int in_dtype,
                 void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace for T tokens, or a negative gemm_status_t (T, H, I, E or
 * topk invalid or unsupported). */
int64_t gemm_moe_workspace(int64_t T, const gemm_moe_t *layer);

/* Host-only argument check of gemm_moe_run (see gemm_validate). */
int gemm_validate_moe(int64_t T, const gemm_moe_t *layer, const void *X, int64_t ldx,
                      const float *logits, int64_t ldl, const void *D, int64_t ldd, int in_dtype,
                      const void *workspace, int64_t workspace_bytes);

/* ============================================ balance of a router's experts
 *
 * The loss that keeps a trained router from using a few experts only, the tokens
 * of each expert, and the loss's gradient.  For T tokens with logits l (T x E),
 * the choice of experts being gemm_moe_run's (the topk largest logits, ties to
 * the lower index, none at -Inf or NaN), over the n tokens that count:
 *
 *   p_te = exp(l_te - lse_t),   lse_t = log sum_e exp(l_te)
 *   c_e  = tokens that chose e,   f_e = c_e / (n topk),   P_e = sum_t p_te / n
 *   loss[1] = E sum_e f_e P_e       (1 when all experts are used alike)
 *   loss[2] = sum_t lse_t^2 / n     (keeps the logits from drifting)
 *   loss[0] = balance * loss[1] + z * loss[2]
 *
 * and, with f held constant (a count has no slope) and g = *dloss (1 if NULL),
 *
 *   D_te = g / n * ( balance E p_te (f_e - sum_j f_j p_tj) + 2 z lse_t p_te ).
 *
 * A token does not count where mask is given and mask[t] is 0, or where all of its
 * logits are -Inf: it adds nothing, and its row of D is 0.  With n == 0 the loss and
 * D are 0.  A counted token with a NaN or +Inf among its logits makes the loss and its
 * own row of D NaN, and no other row.
 *
 *   T            tokens, 0 to 2^31-1
 *   E, topk      1 to 1024 experts, 1 to 32 of them (<= E) for a token
 *   logits, ldl  fp32, row-major, ldl >= E
 *   mask         T bytes on the device, or NULL (every token counts).  A token that
 *                does not count is not read.
 *   loss         3 fp32 values (gemm_moe_balance writes)
 *   counts       E + 1 int32: c_e, then n (gemm_moe_balance writes, _grad reads)
 *   lse          T fp32 values; 0 for a masked token, -Inf for one whose logits all are
 *                (gemm_moe_balance writes, _grad reads)
 *   dloss        one fp32 value on the device, the gradient of loss[0], or NULL (1)
 *   D, ldd       T x E of out_dtype (GEMM_F32, GEMM_F16 or GEMM_BF16), row-major; nothing
 *                outside is written
 *   workspace    device memory of at least gemm_moe_balance_workspace(T, E, topk) bytes,
 *                of any content, owned by the caller, written by the call.  Calls that
 *                may overlap need workspaces of their own.
 * gemm_moe_balance enqueues two kernels, gemm_moe_balance_grad one.  Both allocate
 * nothing, can be captured into a HIP graph, and give the same bits for the same call.
 *
 * Logits of 16-byte aligned lines are read 16 bytes at a time: up to 12 bytes of the padding
 * next to a row's last element too, also past the last row's.
 *
 * Accuracy: softmax and logarithm are fp32 (a p below 2^-126 may be 0); sums of p over tokens are
 * fp32 over up to 32 of them and fp64 beyond, those of lse^2 fp64; D is rounded once.
 *
 * Errors: GEMM_ERR_INVALID_DIM (T < 0 or above 2^31-1, E or topk < 1, topk > E),
 * GEMM_ERR_UNSUPPORTED (E > 1024, topk > 32, out_dtype; a weight that is not finite),
 * GEMM_ERR_INVALID_LD, GEMM_ERR_NULL_PTR, GEMM_ERR_ALIASING (what is written overlapping
 * another argument), GEMM_ERR_SCRATCH_TOO_SMALL, GEMM_ERR_HIP.
 */
int gemm_moe_balance(int64_t T, int64_t E, int64_t topk, const float *logits, int64_t ldl,
                     const uint8_t *mask, float balance, float z, float *loss, int32_t *counts,
                     float *lse, void *workspace, int64_t workspace_bytes, void *stream);
int gemm_moe_balance_grad(int64_t T, int64_t E, int64_t topk, const float *logits, int64_t ldl,
                          const uint8_t *mask, float balance, float z, const int32_t *counts,
                          const float *lse, const float *dloss, void *D, int64_t ldd,
                          int out_dtype, void *stream);

/* Bytes of workspace, or a negative gemm_status_t. */
int64_t gemm_moe_balance_workspace(int64_t T, int64_t E, int64_t topk);

/* Host-only argument checks (see gemm_validate). */
int gemm_validate_moe_balance(int64_t T, int64_t E, int64_t topk, const float *logits, int64_t ldl,
                              const uint8_t *mask, float balance, float z, const float *loss,
                              const int32_t *counts, const float *lse, const void *workspace,
                              int64_t workspace_bytes);
int gemm_validate_moe_balance_grad(int64_t T, int64_t E, int64_t topk, const float *logits,
                                   int64_t ldl, const uint8_t *mask, float balance, float z,
                                   const int32_t *counts, const float *lse, const float *dloss,
                                   const void *D, int64_t ldd, int out_dtype);

/* ===================================================== low-rank adapters
 *
 * Adapters of many requests at once beside a shared projection.  For each token t
 * with a = ids[t],
 *
 *   D(t,:) = C(t,:) + s_a * (x_t A_a^T) B_a^T,
 *
 * and D(t,:) = C(t,:) where ids[t] names no adapter (any value outside [0, adapters)).
 * C is the shared projection's output (e.g. gemm_run's or gemm_run_scaled's D).
 *
 * gemm_lora_t describes the adapters of one projection:
 *   K, N         input and output width, 1 to 2^19
 *   adapters     1 to 2^20
 *   rank         rows kept for each adapter, 1 to 256
 *   A, lda       adapters x rank rows of K elements, lines lda >= K elements apart
 *   B, ldb       adapters x N rows of rank elements, lines ldb >= rank elements apart
 *   ranks        device pointer to one int32 for each adapter, its own rank (0 to rank;
 *                what lies outside is clamped), or NULL (rank for all).  Rows of A and
 *                columns of B from the adapter's rank on are not part of it.
 *   scales       device pointer to one fp32 for each adapter, or NULL (1)
 *
 * gemm_lora_run:
 *   T            tokens, 0 to 2^20
 *   X, ldx       T x K of in_dtype (GEMM_F16 or GEMM_BF16, the type of A and B too)
 *   ids          T int32 on the device, in any order
 *   C, ldc       T x N of out_dtype, row-major, or NULL (C = 0).  C == D with ldc == ldd is
 *                the in-place update; any other overlap is refused.
 *   D, ldd       T x N of out_dtype (GEMM_F32, GEMM_F16 or GEMM_BF16), row-major; nothing
 *                outside is written
 *   workspace    device memory of at least gemm_lora_workspace(T, lora) bytes, of any
 *                content, owned by the caller, written by the call.  A call must not overlap
 *                another one (or a graph's replay) that uses the same workspace, unless the
 *                caller orders them.
 * The call enqueues one kernel (few tokens, rank 32 at most), two, or past 256 tokens three,
 * and allocates nothing, so it can be captured into a HIP graph; which tokens use which
 * adapter is found on the device, and a replay follows the ids of its own time.  Tokens do
 * not touch each other: what an adapter holds (an Inf, a NaN) reaches its own tokens only.
 * The same call gives the same bits.
 *
 * Accuracy: products and sums are fp32, and D is rounded once.  Past 256 tokens the second
 * product takes h = x A^T as a sum of values of in_dtype: two of them for a 16-bit D (16
 * significant bits for bf16, 22 for fp16), three for an fp32 D (24 and 33).  fp16 values are
 * those of h times a power of two that follows the token's largest |h|, so h may lie anywhere
 * in fp32's range, and what is below 2^-38 of that largest value is lost.
 *
 * Speed: 16-byte loads of X and A where both are 16-byte aligned with lines of whole 16
 * bytes, of B alike, and (past 256 tokens) of C and D; element by element otherwise.  With
 * them, up to 14 bytes of the padding next to a row's last element are read, also past the
 * last row's, and never matter.  Up to 256 tokens may use any adapters in any order (a decoding
 * batch).  More of them are taken in tiles of consecutive ones, 64 for A and 32 for B (16 past
 * rank 64), and an adapter's A or B is read once for each tile that it has tokens in: packed
 * prompts.  There, adapters that change from token to token cost that much more (512 tokens on
 * 4096 x 4096, rank 16: 15 us in prompts of 4 adapters, 164 with 32 adapters mixed), and sums
 * that are NaN, which are made again one by one, too.
 *
 * Errors: GEMM_ERR_INVALID_DIM (T < 0; K, N, adapters or rank < 1; K or N > 2^19),
 * GEMM_ERR_UNSUPPORTED (T > 2^20, adapters > 2^20, rank > 256, a dtype not named above),
 * GEMM_ERR_INVALID_LD (a line shorter than its row, or longer than 2^24 elements),
 * GEMM_ERR_NULL_PTR, GEMM_ERR_ALIASING (D or the workspace overlapping another argument),
 * GEMM_ERR_SCRATCH_TOO_SMALL, GEMM_ERR_HIP.
 */
typedef struct {
    int64_t K, N, adapters, rank;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb;
    const int32_t *ranks;
    const float *scales;
} gemm_lora_t;

int gemm_lora_run(int64_t T, const gemm_lora_t *lora, const void *X, int64_t ldx,
                  const int32_t *ids, const void *C, int64_t ldc, void *D, int64_t ldd,
                  int in_dtype, int out_dtype, void *workspace, int64_t workspace_bytes,
                  void *stream);

/* Bytes of workspace for T tokens, or a negative gemm_status_t. */
int64_t gemm_lora_workspace(int64_t T, const gemm_lora_t *lora);

/* Host-only argument check of gemm_lora_run (see gemm_validate). */
int gemm_validate_lora(int64_t T, const gemm_lora_t *lora, const void *X, int64_t ldx,
                       const int32_t *ids, const void *C, int64_t ldc, const void *D, int64_t ldd,
                       int in_dtype, int out_dtype, const void *workspace,
                       int64_t workspace_bytes);

/* ====================================== activation checkpoints in 8 bits
 *
 * Activations kept for the backward pass in 8 bits and a quarter, and what the
 * backward pass does with them.  The format is MXINT8 of the OCP Microscaling
 * Formats specification (version 1.0): 32 consecutive values of a row (the last
 * block of a row may be shorter) share a power of two, one byte S (E8M0), and each
 * value is an int8 Q:
 *
 *   X^(m,k) = 2^(S(m, k/32) - 127) * Q(m,k) / 64.
 *
 * X^ has at most seven significant bits and a power of two, so it is exact in bf16
 * (and in fp16 where X was fp16), and the matrix units multiply it as it is: the
 * rounding of gemm_checkpoint_pack is the only one.
 *   Q, ldq       int8, M x K, row-major, ldq >= K
 *   S, lds       bytes, M x ceil(K / 32), row-major, lds >= ceil(K / 32)
 * Nothing outside the matrices is written.  No call allocates; all can be captured
 * into a HIP graph; calls on different streams do not touch each other.
 *
 * gemm_checkpoint_pack: for each block with a = max |X|,
 *   S = 127 + floor(log2(a)), at least 0 (a = 0: S = 0),
 *   Q = X * 64 / 2^(S - 127), rounded to nearest even, held in [-127, 127].
 * |X^ - X| is at most half a step of 2^(S - 133), or less than a whole one where Q was
 * held back (|X| within a half step of 2^(S - 126)).  A block that holds an Inf or a NaN
 * gets S = 255 and zeros, which stand for NaN.
 *   X, ldx       M x K of in_dtype (GEMM_F16, GEMM_BF16 or GEMM_F32), row-major
 *
 * gemm_checkpoint_unpack: D = X^, rounded once to out_dtype (GEMM_F32, GEMM_F16 or
 * GEMM_BF16; exact but for fp16 values outside its range).
 *
 * gemm_checkpoint_act_grad: D = G * act'(X^), rounded once; G and D of `dtype`, M x K,
 * row-major.  D == G with ldd == ldg is the in-place update.
 *   activation   GEMM_ACT_RELU (D = G for X^ > 0, else 0, whatever G holds; NaN where X^ is),
 *                GEMM_ACT_GELU (Phi(x) + x phi(x)) or GEMM_ACT_SILU (s + x s (1 - s),
 *                s = 1 / (1 + exp(-x)))
 * Between X^ and the rounding everything is fp32: act' is within 1e-6 absolutely, and for
 * X^ < 0, where it goes to 0, within 2^-20 + x^2 2^-24 (SiLU: 2^-20 + |x| 2^-23) of the sum of its
 * two terms' magnitudes (what is below 2^-126 of an exponential may be 0).
 *
 * gemm_checkpoint_wgrad: a linear layer's weight gradient, D = G^T X^ + C:
 *   D(n,k) = sum_m G(m,n) X^(m,k) + C(n,k)
 *   G, ldg       M x N of in_dtype (GEMM_F16 or GEMM_BF16), row-major: the gradient of
 *                the layer's output
 *   C, ldc       N x K of out_dtype, row-major, or NULL (C = 0).  C == D with ldc == ldd
 *                adds up gradients in place; any other overlap is refused.
 *   D, ldd       N x K of out_dtype (GEMM_F32, GEMM_F16 or GEMM_BF16), row-major
 *   workspace    device memory of at least gemm_checkpoint_wgrad_workspace(M, N, K) bytes
 *                (may be 0, then NULL is fine), of any content, owned by the caller,
 *                written by the call.  Calls that may overlap need workspaces of their own.
 * M, the tokens, is the reduction's length; with M == 0, D = C (or 0).  X^ is taken in
 * in_dtype (exact as said above; with GEMM_F16, values past 65504 become Inf, and those below
 * 2^-14 are rounded to steps of 2^-24, which those of an fp16 X are), products are exact and
 * summed in fp32, and D is rounded once.  The same call gives the same bits.
 *
 * Speed: 16-byte accesses where the operands' base pointers and lines are whole 16 bytes
 * (for wgrad G and Q, for the others X, G, D and Q); element by element otherwise.  With
 * them, bytes of the padding next to a row's last element are read (up to 15 past the
 * last row's), and never matter.  wgrad reads S in aligned dwords: up to 3 bytes beside its
 * rows, also before the first.
 *
 * Errors: GEMM_ERR_INVALID_DIM (a dimension negative or above 2^31-1), GEMM_ERR_INVALID_LD
 * (a line shorter than its row, or longer than 2^40 elements), GEMM_ERR_NULL_PTR,
 * GEMM_ERR_UNSUPPORTED (a dtype or activation not named), GEMM_ERR_ALIASING (what is
 * written overlapping another argument), GEMM_ERR_SCRATCH_TOO_SMALL, GEMM_ERR_HIP.
 */
int gemm_checkpoint_pack(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype, void *Q,
                         int64_t ldq, uint8_t *S, int64_t lds, void *stream);
int gemm_checkpoint_unpack(int64_t M, int64_t K, const void *Q, int64_t ldq, const uint8_t *S,
                           int64_t lds, void *D, int64_t ldd, int out_dtype, void *stream);
int gemm_checkpoint_act_grad(int64_t M, int64_t K, const void *Q, int64_t ldq, const uint8_t *S,
                             int64_t lds, const void *G, int64_t ldg, int activation, void *D,
                             int64_t ldd, int dtype, void *stream);
int gemm_checkpoint_wgrad(int64_t M, int64_t N, int64_t K, const void *G, int64_t ldg,
                          const void *Q, int64_t ldq, const uint8_t *S, int64_t lds,
                          const void *C, int64_t ldc, void *D, int64_t ldd, int in_dtype,
                          int out_dtype, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace (possibly 0), or a negative gemm_status_t. */
int64_t gemm_checkpoint_wgrad_workspace(int64_t M, int64_t N, int64_t K);

/* Host-only argument checks (see gemm_validate). */
int gemm_validate_checkpoint_pack(int64_t M, int64_t K, const void *X, int64_t ldx, int in_dtype,
                                  const void *Q, int64_t ldq, const uint8_t *S, int64_t lds);
int gemm_validate_checkpoint_unpack(int64_t M, int64_t K, const void *Q, int64_t ldq,
                                    const uint8_t *S, int64_t lds, const void *D, int64_t ldd,
                                    int out_dtype);
int gemm_validate_checkpoint_act_grad(int64_t M, int64_t K, const void *Q, int64_t ldq,
                                      const uint8_t *S, int64_t lds, const void *G, int64_t ldg,
                                      int activation, const void *D, int64_t ldd, int dtype);
int gemm_validate_checkpoint_wgrad(int64_t M, int64_t N, int64_t K, const void *G, int64_t ldg,
                                   const void *Q, int64_t ldq, const uint8_t *S, int64_t lds,
                                   const void *C, int64_t ldc, const void *D, int64_t ldd,
                                   int in_dtype, int out_dtype, const void *workspace,
                                   int64_t workspace_bytes);

/* ============================================================ autotuning
 *
 * Runtime search over the tile-shape table for one problem signature,
 * cached.  Source: "矩阵乘法优化可视化学习文档", section 6 "常用优化方法总表"
 * (Autotuning row: the best tile differs with M/N/K, dtype and GPU, and is
 * found by search) and section 8 (Autotune: one kernel timed over several
 * block sizes, the fastest kept).
 *
 * gemm_autotune runs the call once per table entry (one untimed run, then
 * `reps` timed runs, clamped to [1, 100]; the minimum counts; an entry more
 * than 2x slower than the best so far stops early), records the fastest
 * entry for the signature (M, N, K, layouts, dtypes, current device; a
 * column-major D is keyed as its transpose, which is what runs), writes it to
 * *config_out (if not NULL; -1 for an empty problem) and leaves D holding the
 * chosen entry's result.  From then on gemm_run / gemm_run_ex with that
 * signature use the recorded entry (gemm_select_config still reports the
 * static choice).  The call synchronises `stream` (HIP events), so it does
 * not belong in a timed region or a graph capture.
 * Arguments and errors as gemm_run_ex, plus: an in-place update (C == D with
 * beta != 0) -> GEMM_ERR_ALIASING, since every candidate run would apply it.
 * The cache is process-wide and guarded by a mutex.
 *
 * gemm_autotune_lookup: the recorded entry for a signature, or -1.
 * gemm_autotune_clear: forget every recorded entry.
 */
int gemm_autotune(int64_t M, int64_t N, int64_t K,
                  const void *A, int64_t lda, int layoutA,
                  const void *B, int64_t ldb, int layoutB,
                  const void *C, int64_t ldc,
                  void *D, int64_t ldd,
                  int in_dtype, int acc_dtype, int out_dtype,
                  int satf, const gemm_epilogue_t *epi, int reps, int *config_out,
                  void *stream);
int gemm_autotune_lookup(int64_t M, int64_t N, int64_t K, int layoutA, int layoutB,
                         int in_dtype, int acc_dtype, int out_dtype, int layoutD);
void gemm_autotune_clear(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBGEMM_H */
