/*
 * gemm_f8 -- products of 8-bit floating-point matrices with a scale for each
 * block of 128, their quantisation, and the rows of layers of experts
 * (sorting tokens by expert and bringing them back).
 *
 * A matrix of 8-bit codes X (e4m3 or e5m2) comes with FP32 scales, one for
 * each block of 128 consecutive numbers along one of its dimensions, or for
 * each 128 x 128 tile; it stands for the numbers code * scale.  The blocks of
 * a product's operands lie along the inner dimension:
 *
 *     C[m,n] = sum_b  sa[m,b] sb[b,n]  sum_{k in block b} A[m,k] B[k,n]
 *
 * with the inner sums on the tensor cores and the outer ones in FP32, and one
 * rounding to C's type.  A block's inner sum is multiplied with one scale and
 * then the other (or, where that is a normal FP32 number, with their product):
 * where the first of these is below 2^-126, digits are lost that a large second
 * scale would have shown, and where it passes FP32's largest number (a scale
 * above 2^89) the result is infinite even if a small second scale would have
 * brought it back.  The last block of a dimension may be shorter.
 *
 * Conventions are those of gemm_f16.h: device pointers on the plan's device,
 * leading dimensions in elements, GEMM_F16_* codes (on an error nothing has
 * been enqueued), calls asynchronous on `stream` and free to be captured into
 * CUDA graphs, one thread and one stream at a time for a plan.  No call here
 * uses memory of the plan's but its status word, so that calls of several
 * plans, and replays of several graphs, never share a workspace.
 */
#ifndef GEMM_F8_H
#define GEMM_F8_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Formats of codes; their largest numbers are 448 and 57344. */
enum { GEMM_F8_E4M3 = 0, GEMM_F8_E5M2 = 1 };

/* Types of what is quantised, of results, and of the experts' rows. */
enum { GEMM_F8_F16 = 0, GEMM_F8_BF16 = 1, GEMM_F8_F32 = 2 };

/* Blocks of a quantisation: 128 numbers along a row, 128 along a column,
 * 128 x 128, or the first two at once from one reading. */
enum { GEMM_F8_ROWS = 0, GEMM_F8_COLUMNS = 1, GEMM_F8_TILES = 2, GEMM_F8_BOTH = 3 };

/*
 * Codes and scales of X, `batch` matrices of rows x cols numbers of `type`.
 * For each block, a = max(2^-100, its largest finite magnitude) and L the
 * format's largest number:
 *     scale = fl(a / L),   code = round(fl(x * fl(L / a)))
 * (fl: to FP32; round: to nearest, ties to even, in the format).  Infinities
 * and NaN become NaN.  Every step is an IEEE operation: results are the same
 * bits for each way of computing them.
 *   X        row r of matrix b at X + b*x_batch + r*ldx; any alignment of its
 *            type (rows on 16-byte boundaries are read faster).
 *   source   NULL, or `rows` entries (batch 1): row r of the result is
 *            row source[r] / choices of X, which has x_rows rows, and 0 where
 *            source[r] is -1 (experts_maps' `source`).  Any other entry
 *            outside [0, x_rows * choices) gives 0 and is reported
 *            (GEMM_F16_ERR_BAD_INDEX).
 *   Q, Q2    codes, rows ldq apart, matrices q_batch: 16-byte aligned
 *            multiples of 16.  Q2: the codes of COLUMNS for BOTH, else unused.
 *   S, S2    scales, contiguous: [batch][rows][ceil(cols/128)] for ROWS,
 *            [batch][ceil(rows/128)][cols] for COLUMNS,
 *            [batch][ceil(rows/128)][ceil(cols/128)] for TILES; for BOTH S is
 *            ROWS' and S2 COLUMNS'.
 *   batch 0 .. 65535, rows 0 .. 2^31 - 1024, cols 1 .. 2^31 - 1024 (batch or rows
 *   0: nothing is enqueued).  Outputs must not overlap X or each other.
 */
int gemm_f8_quantize(gemm_f16_plan_t plan, int blocks, int format, int type, int batch, int rows,
                     int cols, const void *X, int64_t ldx, int64_t x_batch,
                     const int32_t *source, int choices, int x_rows, void *Q, int64_t ldq,
                     int64_t q_batch, float *S, void *Q2, float *S2, gemm_f16_stream_t stream);
int gemm_f8_quantize_validate(int blocks, int format, int type, int batch, int rows, int cols,
                              const void *X, int64_t ldx, int64_t x_batch, const int32_t *source,
                              int choices, int x_rows, const void *Q, int64_t ldq,
                              int64_t q_batch, const float *S, const void *Q2, const float *S2);

/*
 * An operand of a product: a matrix of codes with its scales.
 *   data, ld      row-major storage of the matrix or, with `transposed`, of
 *                 its transpose; 16-byte aligned, ld a multiple of 16.
 *   batch         codes from one matrix to the next (B by expert), a multiple
 *                 of 16.
 *   format        GEMM_F8_E4M3 or GEMM_F8_E5M2; A's and B's may differ.
 *   tiles         0: a scale for each row of A (column of B) and block of the
 *                 inner dimension; 1: for each 128 of them.
 *   s_outer, s_inner, s_batch
 *                 strides of the scales, in elements: along A's rows (B's
 *                 columns) or their 128s, along the inner dimension's blocks,
 *                 and from one matrix to the next.
 */
typedef struct gemm_f8_operand {
    const void *data;
    int64_t ld, batch;
    const float *scales;
    int64_t s_outer, s_inner, s_batch;
    int format, transposed, tiles;
} gemm_f8_operand;

/* Forms of a product. */
enum {
    GEMM_F8_DENSE = 0,
    /* Rows of A and C sorted by expert: those from starts[e] to
     * starts[e+1] - 1 are multiplied with B's matrix e.  A is row-major. */
    GEMM_F8_BY_ROWS = 1,
    /* The inner dimension sorted by expert: C's matrix e is the product of
     * A's columns and B's rows from starts[e] to starts[e+1] - 1, and 0
     * where there are none.  Every start is a multiple of 128. */
    GEMM_F8_BY_INNER = 2
};

/*
 * C = A B, or C += A B with `accumulate` (FP32 C).
 *   M, N, K     A is M x K, B K x N (each matrix), C M x N (each matrix);
 *               M, N >= 0 (0: nothing is enqueued), K >= 0 (0: C is 0), all below
 *               2^31 - 1024.
 *               BY_ROWS: M is the room in A and C; rows past starts[experts]
 *               are set to 0 (left alone with `accumulate`) and rows before
 *               starts[0] are not written.  BY_INNER: K is the room.
 *   experts     1 .. 1024 for the forms by expert, with starts[experts + 1]
 *               on the device; starts that decrease, pass the room or, BY_INNER,
 *               are no multiples of 128 (the end of the room may be none) are
 *               reported (GEMM_F16_ERR_BAD_INDEX).  They make that expert's
 *               matrix NaN (BY_INNER) or leave its rows unspecified (BY_ROWS;
 *               also those of an expert that begins before the end of an earlier
 *               one).  The other experts' rows and matrices are right, and rows
 *               past the last of them 0 (BY_ROWS; nothing is written where every
 *               expert's starts are bad).
 *   C           row-major, of `type`, rows ldc apart, matrices c_batch apart;
 *               its type's alignment (faster on 16-byte rows).  Must not
 *               overlap the operands.
 *   workspace   gemm_f8_workspace(...) bytes (0 for most products) for this
 *               call alone, 16-byte aligned: FP32 partial sums of tiles that
 *               are cut along the inner dimension.  They are added in a fixed
 *               order, so that a call's result is the same bits every time.
 * Returns GEMM_F16_OK, GEMM_F16_ERR_INVALID_ARG, GEMM_F16_ERR_MISALIGNED,
 * GEMM_F16_ERR_SCRATCH_TOO_SMALL (the workspace) or GEMM_F16_ERR_CUDA.
 * GEMM_F16_OPT_TIMEOUT_NS, _SM_LIMIT (both launches of a product with cut tiles;
 * no other call of this header) and _KERNEL_TIMING (the product's kernel, not the
 * join of cut tiles, which takes up to 7 us) apply;
 * GEMM_F16_OPT_FAULT_UNIT names the unit whose first copy is left out.
 */
int gemm_f8_run(gemm_f16_plan_t plan, int form, int M, int N, int K, int experts,
                const int32_t *starts, const gemm_f8_operand *A, const gemm_f8_operand *B, void *C,
                int64_t ldc, int64_t c_batch, int type, int accumulate, void *workspace,
                size_t workspace_bytes, gemm_f16_stream_t stream);
/* Bytes of workspace for these sizes (A's `transposed` decides the kernel
 * too); a call with other sizes needs its own. */
size_t gemm_f8_workspace(gemm_f16_plan_t plan, int form, int M, int N, int K, int experts,
                         int a_transposed);
/* What a call of these sizes launches, on the host and for given facts: SMs,
 * co-resident CTA pairs, GEMM_F16_OPT_SM_LIMIT (0: none).  info[0]: 1 the kernel
 * for few rows, 2 that for many; info[1]: CTAs that share a tile's inner range
 * (1), or parts of a cut tile (2; 1: none is cut); info[2]: CTAs of the product;
 * info[3]: CTAs of the kernel that joins cut tiles (0: there is none).  Returns
 * GEMM_F16_OK or GEMM_F16_ERR_INVALID_ARG. */
int gemm_f8_run_choice(int form, int M, int N, int K, int experts, int a_transposed, int num_sms,
                       int max_pairs, int sm_limit, int info[4]);
int gemm_f8_validate(int form, int M, int N, int K, int experts, const int32_t *starts,
                     const gemm_f8_operand *A, const gemm_f8_operand *B, const void *C,
                     int64_t ldc, int64_t c_batch, int type, int accumulate);

/*
 * Sorting by expert.  experts[i], i = token * choices + choice, names the
 * expert that a token's choice goes to (32-bit integers, or 64-bit with
 * `wide`); the entries are put in order of expert, and within one in order of
 * i, each expert's rows filled up to a multiple of `align`:
 *     starts[0 .. num_experts]   first row of each expert; starts[0] = 0
 *     rows[i]                    entry i's row, or -1 for an entry that is no
 *                                expert's (negative; one >= num_experts is
 *                                also reported, GEMM_F16_ERR_BAD_INDEX)
 *     source[r], r < max_rows    the entry at row r, or -1
 * entries 0 .. 2^26, num_experts 1 .. 1024, align 1 .. 1024, max_rows at least
 * experts_max_rows(entries, num_experts, align).  One launch.
 */
int experts_maps(gemm_f16_plan_t plan, int entries, const void *experts, int wide,
                 int num_experts, int align, int max_rows, int32_t *starts, int32_t *rows,
                 int32_t *source, gemm_f16_stream_t stream);
int experts_maps_validate(int entries, const void *experts, int wide, int num_experts, int align,
                          int max_rows, const int32_t *starts, const int32_t *rows,
                          const int32_t *source);
/* Rows that hold any choice of experts (a multiple of align), or a negative code. */
int64_t experts_max_rows(int entries, int num_experts, int align);

/*
 * Y[r] = X[source[r] / choices], or 0 where source[r] is -1: the tokens' rows
 * in the experts' order.  X has x_rows rows and Y `rows`, of cols numbers;
 * rows ldx, ldy apart.  Entries out of range give 0 and are reported.
 */
int experts_gather(gemm_f16_plan_t plan, int type, int rows, int cols, const void *X, int64_t ldx,
                   int x_rows, int choices, const int32_t *source, void *Y, int64_t ldy,
                   gemm_f16_stream_t stream);

/*
 * Y[t] = sum_j w[t,j] S[rows[t,j]] over the choices with a row, in their
 * order, in FP32, rounded once.  weights: NULL (all 1) or tokens x choices
 * numbers, contiguous, of weights_type (GEMM_F8_F32 or `type`).  S has s_rows
 * rows.  Entries out of range other than -1 are left out and reported.
 */
int experts_combine(gemm_f16_plan_t plan, int type, int tokens, int choices, int cols,
                    const void *S, int64_t lds, int s_rows, const int32_t *rows,
                    const void *weights, int weights_type, void *Y, int64_t ldy,
                    gemm_f16_stream_t stream);

/*
 * The gradients of experts_combine, given that of Y:
 *     dS[r] = w[source[r]] dY[source[r] / choices]   (0 where source[r] is -1)
 *     dw[i] = dY[i / choices] . S[rows[i]]           (0 where rows[i] is -1)
 * dS and dw (contiguous, of weights_type) may each be NULL where not wanted.
 * rows and source are those of one call of experts_maps; S and dS have s_rows
 * rows, the entries of source.
 */
int experts_combine_gradient(gemm_f16_plan_t plan, int type, int tokens, int choices, int cols,
                             const void *dY, int64_t lddy, const void *S, int64_t lds, int s_rows,
                             const int32_t *rows, const int32_t *source, const void *weights,
                             int weights_type, void *dS, int64_t ldds, void *dw,
                             gemm_f16_stream_t stream);

/* Host-only checks of the three calls (tokens and rows may be 0). */
int experts_gather_validate(int type, int rows, int cols, const void *X, int64_t ldx, int x_rows,
                            int choices, const int32_t *source, const void *Y, int64_t ldy);
int experts_combine_validate(int type, int tokens, int choices, int cols, const void *S,
                             int64_t lds, int s_rows, const int32_t *rows, const void *weights,
                             int weights_type, const void *Y, int64_t ldy);
int experts_combine_gradient_validate(int type, int tokens, int choices, int cols, const void *dY,
                                      int64_t lddy, const void *S, int64_t lds, int s_rows,
                                      const int32_t *rows, const int32_t *source,
                                      const void *weights, int weights_type, const void *dS,
                                      int64_t ldds, const void *dw);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F8_H */
