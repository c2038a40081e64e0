/*
 * gemm_gated.h - the gated projections of a feed-forward block in bfloat16:
 * both products, the activation and their product in one kernel, with the
 * backward pass, on one AMD Instinct MI355X (gfx950).
 *
 *     z_gate = x . w_gate + b_gate,   z_up = x . w_up + b_up
 *     h      = act(z_gate) * z_up
 *
 * x has a row per token; the weights are stored [K][N] (GEMM_WEIGHTS_KN) or
 * [N][K] (GEMM_WEIGHTS_NK, one row per output channel).  Sums, biases and the
 * activation are 32-bit floats; h is rounded once.  For training z_gate and
 * z_up are stored too, in floats or rounded to bfloat16 (which takes half the
 * memory and puts a relative error of up to 2^-8 into them).
 *
 * Backward, from dh and the stored z_gate, z_up:
 *
 *     dz_gate = dh * z_up * act'(z_gate),    dz_up = dh * act(z_gate)
 *     dx      = dz_gate . w_gate^T + dz_up . w_up^T       (one sum, rounded once)
 *     dw_gate = x^T . dz_gate,               dw_up = x^T . dz_up
 *     db_gate = sum_rows dz_gate,            db_up = sum_rows dz_up
 *
 * dz is rounded to bfloat16 where it is an operand of dx and dw; the biases'
 * gradients sum the unrounded values.  Sums that several workgroups share are
 * joined in a fixed order (no atomics): equal inputs give equal bits.
 *
 * Activations: GEMM_ACT_NONE (act(z) = z), GEMM_ACT_RELU (its derivative at 0 is
 * 0), GEMM_ACT_GELU (z * Phi(z)), GEMM_ACT_GELU_TANH (its form with tanh) and
 * GEMM_ACT_SILU (z / (1 + exp(-z))), in floats within 1e-5 of their value, or 1e-17
 * where that is more (far out on the negative side), and their derivatives within
 * 1e-5.
 *
 * Status codes and gemm_rs_strerror are those of gemm_rs.h.  All functions
 * are plain C, never throw, abort or print.
 */
#ifndef GEMM_GATED_H
#define GEMM_GATED_H

#include <stdint.h>

#include "gemm_rs.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_ACT_NONE 0
#define GEMM_ACT_RELU 1
#define GEMM_ACT_GELU 2
#define GEMM_ACT_GELU_TANH 3
#define GEMM_ACT_SILU 4

#define GEMM_WEIGHTS_KN 0
#define GEMM_WEIGHTS_NK 1

/*
 * Problem descriptor.
 *   M            most rows (tokens) of a call (a call may have fewer, down to none)
 *   N, K         columns of each projection; row length of x
 *   layout       GEMM_WEIGHTS_KN or GEMM_WEIGHTS_NK, of both weights
 *   act          GEMM_ACT_*
 *   has_bias     1: b_gate[N] and b_up[N] of bias_dtype
 *   bias_dtype   GEMM_RS_BF16 or GEMM_RS_F32 (the biases' gradients are floats)
 *   backward     1: gemm_gated_backward may be called
 *   dw_dtype     GEMM_RS_BF16 or GEMM_RS_F32
 *   accumulate   1: the gradients of weights and biases are added to what their
 *                arrays hold (in float, rounded once)
 *   z_dtype      GEMM_RS_BF16 or GEMM_RS_F32, of z_gate and z_up as stored
 *   ldx, ldw, ldh, ldz, lddh, lddz, lddx, lddw   row strides in elements, 0: the
 *                row length; each serves both arrays of a pair.  So the two weights
 *                (and z's, and gradients) may be halves of one array: side by side
 *                with a stride of twice their row length, or one below the other.
 * Any sizes and element-aligned addresses are accepted.  The kernels load bfloat16
 * operands whose row lengths, strides and addresses are multiples of 8 elements
 * (16 bytes).  An operand of another row length or stride is copied to padded rows
 * first, in memory that the plan holds (x, the weights, dz; none if they would come
 * to more than 8 GiB).  One that only its address keeps from it, or without room
 * for its copy, takes a kernel that is 2 to 5 times as long.  Up to 16 rows with
 * weights [N][K] (or dx of weights [K][N]) are read at any address and stride; up to
 * 8 without any copy.
 */
typedef struct gemm_gated_desc {
    int64_t M, N, K;
    int32_t layout, act;
    int32_t has_bias, bias_dtype;
    int32_t backward, dw_dtype;
    int32_t accumulate, z_dtype;
    int64_t ldx, ldw, ldh, ldz;
    int64_t lddh, lddz, lddx, lddw;
} gemm_gated_desc_t;

typedef struct gemm_gated_plan_s *gemm_gated_plan_t;

/* Introspection: bytes of device memory that the plan holds. */
typedef struct gemm_gated_info {
    int64_t workspace_bytes;
} gemm_gated_info_t;

/*
 * gemm_gated_plan: validate and allocate.  Returns OK, INVALID_ARG (NULL
 * pointers, M, N or K < 1, unknown layout, act or type, flags other than 0/1,
 * strides below the row length), UNSUPPORTED (M above
 * 2^31-1025, N, K or strides of 2^23 or more, a grid over 2^31-1) or HIP.
 * Rejected before any HIP call.
 */
GEMM_RS_API int gemm_gated_plan(const gemm_gated_desc_t *desc, gemm_gated_plan_t *out);

/*
 * gemm_gated_run: the forward for `rows` rows (0..desc.M), enqueued on
 * `stream`; no host synchronisation, no allocation.
 *   x               [rows][ldx]
 *   w_gate, w_up    [K][ldw] or [N][ldw]
 *   b_gate, b_up    [N] (has_bias; NULL without)
 *   h               [rows][ldh], or NULL where only z is wanted
 *   z_gate, z_up    [rows][ldz], or both NULL (nothing is stored for backward)
 * No output may overlap an input or another output.  With rows == 0 nothing is
 * enqueued, and arrays of rows may be NULL, as arrays without elements are.
 * One plan must not run on two streams at once (its workspace).
 * Returns OK, INVALID_ARG (a missing or superfluous pointer, an address not
 * aligned to its element, rows out of range, another device) or HIP.
 */
GEMM_RS_API int gemm_gated_run(gemm_gated_plan_t plan, const void *x, const void *w_gate, const void *w_up,
                               const void *b_gate, const void *b_up, void *h, void *z_gate, void *z_up,
                               int64_t rows, void *stream);

/*
 * gemm_gated_backward: the gradients for `rows` rows (0..desc.M).
 *   dh               [rows][lddh]
 *   z_gate, z_up     [rows][ldz], as the forward stored them
 *   dz_gate, dz_up   [rows][lddz] bfloat16; they may be bfloat16 z_gate and z_up
 *                    themselves, in place, if the strides agree
 *   dx               [rows][lddx], or NULL
 *   dw_gate, dw_up   shaped as the weights, of dw_dtype, or both NULL
 *   db_gate, db_up   [N] floats, or both NULL (NULL without has_bias)
 * x may be NULL without dw, the weights without dx.  With rows == 0 the gradients
 * of weights and biases are zeros (with `accumulate` nothing is added), and
 * arrays of rows may be NULL.  But for dz in place of z no output may overlap an
 * input or another output.  One plan must not run on two streams at once (its
 * workspace).  Returns as gemm_gated_run, and INVALID_ARG for dz in place of z that
 * is float or has another stride.
 */
GEMM_RS_API int gemm_gated_backward(gemm_gated_plan_t plan, const void *dh, const void *x, const void *w_gate,
                                    const void *w_up, const void *z_gate, const void *z_up, void *dz_gate,
                                    void *dz_up, void *dx, void *dw_gate, void *dw_up, void *db_gate, void *db_up,
                                    int64_t rows, void *stream);

GEMM_RS_API int gemm_gated_query(gemm_gated_plan_t plan, gemm_gated_info_t *info);

/* Free the workspace (synchronise first).  NULL is OK. */
GEMM_RS_API int gemm_gated_destroy(gemm_gated_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_GATED_H */
