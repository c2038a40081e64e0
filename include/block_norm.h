/*
 * block_norm.h - the norms before and after a transformer block, fused with
 * the block's gate and the residual scale, forward and backward, on one
 * AMD Instinct MI355X (gfx950).
 *
 * For each row of a rank's row chunk (the rows the reduce-scatter of
 * gemm_rs.h leaves on it), with y the block's output, x the residual stream
 * and o = weight_offset:
 *
 *     z  = y * r2 * (o + w_post),    r2 = 1/sqrt(mean(y*y) + eps_post)
 *     x' = res_scale * x + gate * z
 *     u  = x' * r1 * (o + w_pre),    r1 = 1/sqrt(mean(x'*x') + eps_pre)
 *
 * x' is the new residual stream, u the next block's input.  u can be
 * written as 8-bit integers with one scale per row (the input of gemm_q8.h,
 * whose rows are padded with zeros to a multiple of 16).  Sums and statistics are 32-bit floats; u is computed from
 * the unrounded x'.
 *
 * Backward, from dx' (gradient of the stream after this point) and du:
 *
 *     a = du * (o + w_pre),  xh = x' * r1,  yh = y * r2
 *     D = dx' + r1 * (a - xh * mean(a * xh)),     dx = res_scale * D
 *     b = D * gate * (o + w_post)
 *     dy = r2 * (b - yh * mean(b * yh))
 *     dw_pre = sum_rows du * xh,     dw_post = sum_rows D * gate * yh
 *     dgate  = sum over the gate's rows of D * z
 *
 * with x' as the forward stored it.  r1 and r2 are recomputed from the rows
 * the backward reads anyway, so the forward saves no statistics.  The sums
 * over rows are taken in a fixed order (no atomics): equal inputs give equal
 * bits.
 *
 * Status codes and gemm_rs_strerror are those of gemm_rs.h.  All functions
 * are plain C, never throw, abort or print.
 */
#ifndef BLOCK_NORM_H
#define BLOCK_NORM_H

#include <stdint.h>

#include "gemm_rs.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Problem descriptor.  Element types are GEMM_RS_BF16 or GEMM_RS_F32.
 *   rows           most rows of a call (a call may have fewer, down to none)
 *   cols           row length, 1..16384
 *   dtype          type of y, u, du, dy
 *   stream_dtype   type of x, x', dx', dx
 *   param_dtype    type of w_post, gate, w_pre (their gradients are floats)
 *   has_y          1: as above.  0: no block (x' = x, only u is computed)
 *   post           1: the norm after the block; 0: z = y
 *   pre            1: the next norm, u; 0: no u (has_y must be 1)
 *   quant          1: u is int8 with a scale per row (dtype says nothing of u)
 *   backward       1: block_norm_backward may be called (allocates its
 *                  workspace); not with quant
 *   rows_per_gate  0: no gate (gate = 1); else row i uses gate row
 *                  i / rows_per_gate of gate[ceil(rows/rows_per_gate)][cols]:
 *                  one vector (rows_per_gate >= rows), one per sample, or
 *                  one per token (1)
 *   ld_*           row strides in elements, 0: cols.  ld_x for x and ld_dx
 *                  for dx, ld_x_out for x', and so on.
 *   res_scale, weight_offset, eps_post, eps_pre   finite; eps >= 0
 *   pad            must be 0
 * Any size, stride and element-aligned address is accepted; rows whose
 * lengths, strides and addresses are all multiples of 8 elements (16 bytes)
 * are faster (8192 rows of 8192 columns forward 98 us, of 8191 116; backward 168
 * and 214).
 */
typedef struct block_norm_desc {
    int64_t rows, cols;
    int32_t dtype, stream_dtype, param_dtype;
    int32_t has_y, post, pre, quant, backward;
    int64_t rows_per_gate;
    int64_t ld_x, ld_y, ld_x_out, ld_u;
    int64_t ld_dx_out, ld_du, ld_dx, ld_dy;
    float res_scale, weight_offset, eps_post, eps_pre;
    int32_t pad;
} block_norm_desc_t;

typedef struct block_norm_plan_s *block_norm_plan_t;

/* Introspection: gate rows of a full call and the backward's workspace. */
typedef struct block_norm_info {
    int64_t gate_rows;
    int64_t workspace_bytes;
} block_norm_info_t;

/*
 * block_norm_plan: validate and allocate.  Returns OK, INVALID_ARG (NULL
 * pointers, rows or cols < 1, a stride below cols, unknown types, flags
 * other than 0/1, post or a gate without has_y, neither has_y nor pre,
 * quant without pre, quant with backward, non-finite scalars, pad),
 * UNSUPPORTED (cols above 16384, rows or rows_per_gate of 2^31 or more,
 * strides of 2^31 or more) or HIP.  Rejected before any HIP call.
 */
GEMM_RS_API int block_norm_plan(const block_norm_desc_t *desc, block_norm_plan_t *out);

/*
 * block_norm_run: the forward for `rows` rows (0..desc.rows), enqueued on
 * `stream`; no host synchronisation, no allocation.
 *   x       [rows][ld_x];  x_out [rows][ld_x_out] (has_y; NULL without; may
 *           be x itself if the strides agree)
 *   y, w_post, gate, w_pre   as the descriptor has them, NULL where it has not
 *   u       [rows][ld_u] (pre; NULL without): dtype, or int8 with quant, where
 *           columns cols..ceil(cols/16)*16 are zeros if ld_u holds them
 *   u_scale [rows] floats (quant; NULL without): u ~ u_int8 * u_scale, with
 *           u_scale = max|u| / 127, and NaN for a row with a NaN or infinity
 * Other than x_out = x, no output may overlap an input or another output.
 * With rows == 0 nothing is enqueued, and every array of rows (gate among
 * them) may be NULL, as arrays without elements are.
 * Returns OK, INVALID_ARG (a missing or superfluous pointer, an address not
 * aligned to its element, rows out of range, another device) or HIP.
 */
GEMM_RS_API int block_norm_run(block_norm_plan_t plan, const void *x, const void *y,
                               const void *w_post, const void *gate, const void *w_pre,
                               void *x_out, void *u, void *u_scale, int64_t rows, void *stream);

/*
 * block_norm_backward: the gradients for `rows` rows (0..desc.rows).
 *   dx_out  gradient of x' [rows][ld_dx_out]; NULL stands for zeros (pre only)
 *   du      [rows][ld_du] (pre; NULL without)
 *   x_out   x' as the forward stored it (x itself without has_y), row stride
 *           ld_x_out (pre; NULL without)
 *   dx      [rows][ld_dx];  dy [rows][ld_dy] (has_y)
 *   dw_post, dw_pre   [cols] floats;  dgate [gate rows][cols] floats, of
 *           which a call writes those of its rows
 * The gradients of parameters are written, not added to; with rows == 0
 * dw_post and dw_pre are zeros, dgate has no rows, and every pointer but
 * w_post, w_pre, dw_post and dw_pre may be NULL.  No output may overlap an
 * input or another output.
 * One plan's backward must not run on two streams at once (its workspace).
 */
GEMM_RS_API int block_norm_backward(block_norm_plan_t plan, const void *dx_out, const void *du,
                                    const void *x_out, const void *y, const void *w_post,
                                    const void *gate, const void *w_pre, void *dx, void *dy,
                                    void *dw_post, void *dgate, void *dw_pre, int64_t rows,
                                    void *stream);

GEMM_RS_API int block_norm_query(block_norm_plan_t plan, block_norm_info_t *info);

/* Free the workspace (synchronise first).  NULL is OK. */
GEMM_RS_API int block_norm_destroy(block_norm_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* BLOCK_NORM_H */
