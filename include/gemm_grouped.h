/*
 * gemm_grouped.h - bfloat16 matrix products grouped by expert, with group
 * sizes that only the device knows, forward and both gradients, on one AMD
 * Instinct MI355X (gfx950).
 *
 * Rows are sorted by expert; expert e has rows [offsets[e], offsets[e+1]).
 * Three forms, each one launch over all experts:
 *
 *   GEMM_GROUPED_NN   C[i] = A[i] . B_e      A [rows][K], B [E][K][N], C [rows][N]
 *   GEMM_GROUPED_NT   C[i] = A[i] . B_e^T    A [rows][K], B [E][N][K], C [rows][N]
 *   GEMM_GROUPED_TN   C_e  = A_e^T . B_e     A [rows][K], B [rows][N], C [E][K][N]
 *
 * For a layer y = x . W_e with W [E][K][N]: the product is NN, the
 * gradient of x is NT (A = dy, B = W), the gradient of W is TN (A = x,
 * B = dy).  For weights stored [E][N][K] the first two swap and the last
 * takes (dy, x).  Accumulation is in 32-bit floats, rounded once to the
 * output type.
 *
 * NN and NT write the rows of the groups only; a row that is in no group is
 * left as it is, and its row of A is not used.  TN writes every C_e: zeros
 * for an expert without rows (nothing is added with `accumulate`).
 *
 * Status codes and gemm_rs_strerror are those of gemm_rs.h.  All functions
 * are plain C, never throw, abort or print.
 */
#ifndef GEMM_GROUPED_H
#define GEMM_GROUPED_H

#include <stdint.h>

#include "gemm_rs.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_GROUPED_NN 0
#define GEMM_GROUPED_NT 1
#define GEMM_GROUPED_TN 2

/*
 * Problem descriptor.
 *   M           most rows of a call, all experts together
 *   N, K        as above
 *   E           experts, 1..1024
 *   op          GEMM_GROUPED_NN, _NT or _TN
 *   out_dtype   GEMM_RS_BF16 or GEMM_RS_F32 (of C; A and B are bfloat16)
 *   accumulate  TN only, 1: C_e += A_e^T . B_e (added in float, rounded once)
 *   lda, ldb, ldc   row strides in elements, 0: the row length.  One expert's
 *               B (NN, NT) or C (TN) lies K (or N) rows of the stride
 *               after the one before.
 *   pad         must be 0
 * Any sizes and element-aligned addresses are accepted.  Sizes, strides and
 * addresses that are all multiples of 8 elements (16 bytes; ldc of floats of 4)
 * take the kernels with direct loads to shared memory, others, also where C
 * alone is not aligned, a kernel that takes 2 to 3.5 times as long (even groups,
 * 8000 rows, 64 experts of 4095 x 1791: 450 us, of 4096 x 1792: 190; 16384 rows, 8
 * experts of 4095 x 3583: 1.4 ms, of 4096 x 3584: 0.4).
 */
typedef struct gemm_grouped_desc {
    int64_t M, N, K;
    int32_t E, op;
    int32_t out_dtype, accumulate;
    int64_t lda, ldb, ldc;
    int64_t pad;
} gemm_grouped_desc_t;

typedef struct gemm_grouped_plan_s *gemm_grouped_plan_t;

/* Introspection: bytes of device memory that the plan holds. */
typedef struct gemm_grouped_info {
    int64_t workspace_bytes;
} gemm_grouped_info_t;

/*
 * gemm_grouped_plan: validate and allocate.  Returns OK, INVALID_ARG (NULL
 * pointers, M, N, K or E < 1, unknown op or type, accumulate other than 0/1
 * or without TN, strides below the row length, pad), UNSUPPORTED (E above
 * 1024, M above 2^31-1025, N, K or strides of 2^23 or more, a grid over 2^31-1)
 * or HIP.  Rejected before any HIP call.
 */
GEMM_RS_API int gemm_grouped_plan(const gemm_grouped_desc_t *desc, gemm_grouped_plan_t *out);

/*
 * gemm_grouped_run: one pass over `rows` rows (0..desc.M), enqueued on
 * `stream`; no host synchronisation, no allocation.
 *   offsets  int32 [E+1] on the device, non-decreasing, within 0..rows.
 *            Other values are clipped to that (no access leaves the
 *            arrays) and reported by gemm_grouped_status.
 *   C        may not overlap an input
 * With rows == 0 NN and NT enqueue nothing (and look at no offsets), TN writes
 * zeros (with `accumulate` nothing); arrays of rows (A, C of NN and NT, B of TN)
 * may be NULL then, as arrays without elements are.
 * One plan of TN must not run on two streams at once (its workspace).
 * Returns OK, INVALID_ARG (NULL or misaligned pointers, rows out of range,
 * another device) or HIP.
 */
GEMM_RS_API int gemm_grouped_run(gemm_grouped_plan_t plan, const void *A, const void *B,
                                 const void *offsets, void *C, int64_t rows, void *stream);

/*
 * gemm_grouped_status: synchronise `stream`, return the error that a run
 * recorded since the last call (OK, or PROTOCOL for offsets that had to be
 * clipped, with detail {code, expert, offsets[e], offsets[e+1]} of one such
 * expert of the first such run), and clear it.  After an
 * error the outputs of that run are undefined.
 */
GEMM_RS_API int gemm_grouped_status(gemm_grouped_plan_t plan, void *stream, int32_t *detail4);

GEMM_RS_API int gemm_grouped_query(gemm_grouped_plan_t plan, gemm_grouped_info_t *info);

/* Free the plan (synchronise first).  NULL is OK. */
GEMM_RS_API int gemm_grouped_destroy(gemm_grouped_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_GROUPED_H */
