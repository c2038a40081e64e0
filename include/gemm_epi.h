/*
 * gemm_epi.h - a bfloat16 matrix product with bias, activation and residual in
 * its epilogue, with the backward pass, on one AMD Instinct MI355X (gfx950).
 *
 *     z = x . w + bias
 *     y = act(z) + r
 *
 * x has a row per token; w is stored [K][N] (GEMM_WEIGHTS_KN) or [N][K]
 * (GEMM_WEIGHTS_NK, one row per output channel).  It is the down projection of
 * a feed-forward block (bias, and the residual stream as r) and the up
 * projection of one without gate (bias and activation).  The sum and what follows
 * it are 32-bit floats; y is rounded once.  For training z is stored too, in floats
 * or rounded to bfloat16.
 *
 * Backward, from dy and the stored z:
 *
 *     dz = dy * act'(z)
 *     dx = dz . w^T,   dw = x^T . dz,   dbias = sum_rows dz
 *
 * and the gradient of r is dy.  dz is rounded to bfloat16 where it is an operand
 * of dx and dw; dbias sums the unrounded values.  Sums that several workgroups
 * share are joined in a fixed order (no atomics): equal inputs give equal bits.
 *
 * Activations and layouts are those of gemm_gated.h; status codes and
 * gemm_rs_strerror those of gemm_rs.h.  All functions are plain C, never throw,
 * abort or print.
 */
#ifndef GEMM_EPI_H
#define GEMM_EPI_H

#include <stdint.h>

#include "gemm_gated.h"
#include "gemm_rs.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Problem descriptor.
 *   M             most rows (tokens) of a call (a call may have fewer, down to none)
 *   N, K          columns of y; row length of x
 *   layout, act   GEMM_WEIGHTS_*, GEMM_ACT_*
 *   out_dtype     GEMM_RS_BF16 or GEMM_RS_F32, of y, r and dy
 *   has_bias      1: bias[N] of bias_dtype (its gradient is floats)
 *   has_residual  1: r
 *   backward      1: gemm_epi_backward may be called
 *   dw_dtype      GEMM_RS_BF16 or GEMM_RS_F32
 *   accumulate    1: dw and dbias are added to what their arrays hold (in float,
 *                 rounded once)
 *   z_dtype       GEMM_RS_BF16 or GEMM_RS_F32, of z as stored
 *   ldx, ldw, ldr, ldy, ldz, lddy, lddz, lddx, lddw   row strides in elements, 0:
 *                 the row length
 * Any sizes and element-aligned addresses are accepted; which are faster is said
 * in gemm_gated.h.
 */
typedef struct gemm_epi_desc {
    int64_t M, N, K;
    int32_t layout, act;
    int32_t out_dtype, has_bias;
    int32_t bias_dtype, has_residual;
    int32_t backward, dw_dtype;
    int32_t accumulate, z_dtype;
    int64_t ldx, ldw, ldr, ldy, ldz;
    int64_t lddy, lddz, lddx, lddw;
} gemm_epi_desc_t;

typedef struct gemm_epi_plan_s *gemm_epi_plan_t;

/* Introspection: bytes of device memory that the plan holds. */
typedef struct gemm_epi_info {
    int64_t workspace_bytes;
} gemm_epi_info_t;

/*
 * gemm_epi_plan: validate and allocate.  Returns OK, INVALID_ARG (NULL pointers,
 * M, N or K < 1, unknown layout, act or type, flags other than 0/1, strides below
 * the row length), UNSUPPORTED (M above 2^31-1025, N, K or
 * strides of 2^23 or more, a grid over 2^31-1) or HIP.  Rejected before any HIP
 * call.
 */
GEMM_RS_API int gemm_epi_plan(const gemm_epi_desc_t *desc, gemm_epi_plan_t *out);

/*
 * gemm_epi_run: the forward for `rows` rows (0..desc.M), enqueued on `stream`; no
 * host synchronisation, no allocation.
 *   x      [rows][ldx];   w [K][ldw] or [N][ldw]
 *   bias   [N] (has_bias; NULL without)
 *   r      [rows][ldr] (has_residual; NULL without)
 *   y      [rows][ldy]; it may be r itself, in place, if the strides agree
 *   z      [rows][ldz] of z_dtype, or NULL (nothing is stored for backward)
 * But for y in place of r no output may overlap an input or another output.  With
 * rows == 0 nothing is enqueued, and arrays of rows may be NULL, as arrays without
 * elements are.  One plan must not run on two streams at once (its workspace).
 * Returns OK, INVALID_ARG (a missing or superfluous pointer, an address not
 * aligned to its element, rows out of range, another device, an output in place of
 * an input of another stride or element size) or HIP.
 */
GEMM_RS_API int gemm_epi_run(gemm_epi_plan_t plan, const void *x, const void *w, const void *bias, const void *r,
                             void *y, void *z, int64_t rows, void *stream);

/*
 * gemm_epi_backward: the gradients for `rows` rows (0..desc.M).
 *   dy     [rows][lddy] of out_dtype
 *   z      [rows][ldz], as the forward stored it; NULL with GEMM_ACT_NONE
 *   dz     [rows][lddz] bfloat16; it may be a bfloat16 z or dy itself, in place, if
 *          the strides agree.  NULL with GEMM_ACT_NONE and a bfloat16 dy, which is
 *          dz then (with row stride lddy)
 *   dx     [rows][lddx] bfloat16, or NULL
 *   dw     shaped as w, of dw_dtype, or NULL
 *   dbias  [N] floats, or NULL (NULL without has_bias)
 * x may be NULL without dw, w without dx.  With rows == 0 dw and dbias are zeros
 * (with `accumulate` nothing is added), and arrays of rows may be NULL.  But for dz
 * in place no output may overlap an input or another output.  One plan must not
 * run on two streams at once (its workspace).
 */
GEMM_RS_API int gemm_epi_backward(gemm_epi_plan_t plan, const void *dy, const void *x, const void *w, const void *z,
                                  void *dz, void *dx, void *dw, void *dbias, int64_t rows, void *stream);

GEMM_RS_API int gemm_epi_query(gemm_epi_plan_t plan, gemm_epi_info_t *info);

/* Free the workspace (synchronise first).  NULL is OK. */
GEMM_RS_API int gemm_epi_destroy(gemm_epi_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_EPI_H */
