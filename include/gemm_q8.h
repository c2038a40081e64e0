/*
 * gemm_q8.h - matrix product in 8-bit integers with a scale for each token
 * and each channel, and the quantisation of its activations, on one AMD
 * Instinct MI355X (gfx950).
 *
 *     D[m][n] = (sum_k a[m][k] * w[n][k]) * a_scale[m] * w_scale[n] + bias[n]
 *
 * a: tokens as rows of int8; w: one row of int8 per output channel (so both
 * operands are contiguous along the contraction).  The sum is exact in 32
 * bits (K < 2^17); it is converted to float (rounded to nearest above
 * 2^24), multiplied by a_scale, then w_scale, and the bias is added with a
 * fused multiply-add; the result is rounded once to the output type.
 *
 * gemm_q8_quantize makes a and a_scale from bfloat16 or float rows:
 *     a_scale[m] = max_k |x[m][k]| / 127
 *     a[m][k]    = round_to_nearest_even(x[m][k] * (127 * (1 / max_k |x[m][k]|)))
 * each step in 32-bit floats, rounded to nearest.  A row of zeros gets scale
 * 0 and zeros; a row with a NaN or an infinity gets scale NaN and zeros, so
 * its products are NaN.
 *
 * Status codes and gemm_rs_strerror are those of gemm_rs.h.  All functions
 * are plain C, never throw, abort or print.
 */
#ifndef GEMM_Q8_H
#define GEMM_Q8_H

#include <stdint.h>

#include "gemm_rs.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Problem descriptor.
 *   M          most rows (tokens) of a call; N channels; K contraction,
 *              a multiple of 16 below 2^17 (pad the rows of a or of w with
 *              zeros up to it: gemm_q8_quantize does, and the block norm's
 *              int8 output does where its row stride has the room)
 *   lda, ldw   row strides in bytes, multiples of 16, 0: K
 *   ldd        row stride of D in elements, 0: N
 *   out_dtype  GEMM_RS_BF16 or GEMM_RS_F32
 *   has_bias   1: bias[N] floats
 */
typedef struct gemm_q8_desc {
    int64_t M, N, K;
    int64_t lda, ldw, ldd;
    int32_t out_dtype;
    int32_t has_bias;
} gemm_q8_desc_t;

typedef struct gemm_q8_plan_s *gemm_q8_plan_t;

/* Introspection: bytes of device memory that the plan holds. */
typedef struct gemm_q8_info {
    int64_t workspace_bytes;
} gemm_q8_info_t;

/*
 * gemm_q8_plan: validate (and allocate).  Returns OK, INVALID_ARG (NULL
 * pointers, M, N or K < 1, strides below the row length, unknown type,
 * has_bias other than 0/1), UNSUPPORTED (K % 16, lda % 16, ldw % 16, K of
 * 2^17 or more, M or N of 2^31 or more, strides of 2^23 or more) or HIP.
 * Rejected before any HIP call.
 */
GEMM_RS_API int gemm_q8_plan(const gemm_q8_desc_t *desc, gemm_q8_plan_t *out);

/*
 * gemm_q8_run: one product over `rows` rows (0..desc.M), enqueued on
 * `stream`; no host synchronisation, no allocation.
 *   a       int8 [rows][lda], 16-byte aligned;   a_scale float [rows]
 *   w       int8 [N][ldw], 16-byte aligned;      w_scale float [N]
 *   bias    float [N], NULL without has_bias
 *   D       [rows][ldd] of out_dtype, element-aligned; it may not overlap
 *           an input
 * With rows == 0 nothing is enqueued, and a, a_scale and D may be NULL, as
 * arrays without elements are.
 * Returns OK, INVALID_ARG (missing, superfluous or misaligned pointers, rows
 * out of range, another device) or HIP (also for more than about
 * 2^28 channels, whose workgroups have more threads than one launch).
 */
GEMM_RS_API int gemm_q8_run(gemm_q8_plan_t plan, const void *a, const void *a_scale,
                            const void *w, const void *w_scale, const void *bias, void *D,
                            int64_t rows, void *stream);

/*
 * gemm_q8_quantize: rows x cols of `dtype` (row stride ldx elements) to int8
 * rows of stride ldq bytes and one float scale per row; columns
 * cols..ceil(cols/16)*16 of the output are zeros (ldq holds them).  Enqueued
 * on `stream`.  rows may be 0, and x, q and scale NULL then; q and scale may
 * not overlap x.  Returns OK, INVALID_ARG (NULL or misaligned pointers: x to
 * its element; rows < 0, cols < 1, ldx < cols, ldq below ceil(cols/16)*16,
 * unknown type), UNSUPPORTED (cols of 2^17 or more, rows or strides of 2^31 or
 * more) or HIP.
 */
GEMM_RS_API int gemm_q8_quantize(const void *x, int32_t dtype, int64_t rows, int64_t cols,
                                 int64_t ldx, void *q, int64_t ldq, void *scale, void *stream);

GEMM_RS_API int gemm_q8_query(gemm_q8_plan_t plan, gemm_q8_info_t *info);

/* Free the plan (synchronise first).  NULL is OK. */
GEMM_RS_API int gemm_q8_destroy(gemm_q8_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_Q8_H */
