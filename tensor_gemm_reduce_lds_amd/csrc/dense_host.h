// Host side that the gated projections and the product with epilogue share:
// checks, the plan's memory, and the backward pass.
#pragma once

#include <stdlib.h>

#include "dense.h"

namespace gemm_rs {
namespace ffn {

// most rows: the last step of 64 that is begun (some are loaded ahead) ends
// within 32 bits
constexpr int64_t kDenseMaxRows = INT32_MAX - 1024;

inline bool flag(int32_t v) { return v == 0 || v == 1; }
// Whether an output may be `in` itself: not where its elements are of another size or
// its rows lie elsewhere, since others would be overwritten before they are read.
inline bool in_place_ok(const void *out, const void *in, bool same_size, int64_t rows, int64_t ld_out, int64_t ld_in) {
    return !out || out != in || (same_size && (ld_out == ld_in || rows <= 1));
}
inline bool stride_ok(int64_t ld, int64_t cols) { return ld >= 0 && (ld == 0 || ld >= cols); }

// What both plans are made of.  Strides are filled in; ldd: of dz as an operand.
struct DenseSizes {
    int64_t M, N, K;
    int32_t layout, act, arrays, backward, sums, dw_f32;      // sums: a bias and its gradient
    int64_t ldx, ldw, ldd;
};
inline int check_sizes(const DenseSizes &d) {
    if (d.M < 1 || d.N < 1 || d.K < 1 || d.act < 0 || d.act >= kActs || (d.layout != GEMM_WEIGHTS_KN && d.layout != GEMM_WEIGHTS_NK))
        return GEMM_RS_ERR_INVALID_ARG;
    return GEMM_RS_OK;
}
inline int check_limits(const DenseSizes &d, const int64_t *ld, int n) {
    if (d.M > kDenseMaxRows || d.N >= kDenseMaxStride || d.K >= kDenseMaxStride) return GEMM_RS_ERR_UNSUPPORTED;
    for (int i = 0; i < n; ++i)
        if (ld[i] >= kDenseMaxStride) return GEMM_RS_ERR_UNSUPPORTED;
    // most workgroups of the narrow kernel, which has the smallest tiles
    const int64_t tm = (d.M + 63) / 64, tn = (d.N + 63) / 64, tk = (d.K + 63) / 64;
    if (tm * tn > INT32_MAX || (d.backward && (tm * tk > INT32_MAX || tk * tn * d.arrays > INT32_MAX))) return GEMM_RS_ERR_UNSUPPORTED;
    return GEMM_RS_OK;
}

// Memory of a plan on the current device: what sums of parts need (a plan's
// launches come one after another, so all share it), and room for padded copies of
// operands whose sizes or strides the kernels with direct loads do not take.
struct DenseMemory {
    int device;
    char *base;                       // or null
    int64_t bytes, slot_bytes;
    float *slots;
    uint16_t *x, *w[2], *dz[2];       // or null
};
constexpr int64_t kMostCopies = int64_t(8) << 30;     // more are not made: the narrow kernel runs

inline int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
inline bool allocate(DenseMemory *m, const DenseSizes &d) {
    const bool kn = d.layout == GEMM_WEIGHTS_KN;
    int64_t most = dense_slots(d.M, d.N, d.K, d.arrays, kn);
    if (d.backward) {
        const int64_t more[] = {dense_slots(d.M, d.K, d.arrays * d.N, 1, !kn),
                                dense_tn_slots(d.M, kn ? d.K : d.N, kn ? d.N : d.K, d.arrays, d.dw_f32 ? 4 : 2),
                                d.sums ? activation_gradient_slots(d.M, d.N, d.arrays) : 0};
        for (int64_t b : more)
            if (b > most) most = b;
    }
    m->slot_bytes = (most + 255) / 256 * 256;
    const int64_t w_rows = kn ? d.K : d.N, w_cols = kn ? d.N : d.K;
    // (a plan for few rows may need none)
    const bool forward = !dense_as_it_is(d.M, d.K, kn), of_x = forward || d.backward;
    const bool of_w = forward || (d.backward && !dense_as_it_is(d.M, d.N, !kn));
    int64_t x = of_x && (d.K % 8 || d.ldx % 8) ? d.M * up8(d.K) * 2 : 0, w = of_w && (w_cols % 8 || d.ldw % 8) ? w_rows * up8(w_cols) * 2 : 0;
    int64_t dz = d.backward && (d.N % 8 || d.ldd % 8) ? d.M * up8(d.N) * 2 : 0;
    // (rows and columns are below 2^31 and 2^23, so this does not overflow)
    if (x + d.arrays * (w + dz) > kMostCopies) x = w = dz = 0;
    for (int64_t *b : {&x, &w, &dz}) *b = (*b + 255) / 256 * 256;
    m->bytes = m->slot_bytes + x + d.arrays * (w + dz);
    if (own(hipGetDevice(&m->device)) != hipSuccess) return false;
    if (m->bytes == 0) return true;
    if (own(hipMalloc((void **)&m->base, (size_t)m->bytes)) != hipSuccess) return false;
    m->slots = (float *)m->base;
    char *at = m->base + m->slot_bytes;
    auto take = [&](uint16_t **to, int64_t bytes) {
        *to = bytes ? (uint16_t *)at : nullptr;
        at += bytes;
    };
    take(&m->x, x);
    for (int i = 0; i < d.arrays; ++i) take(&m->w[i], w);
    for (int i = 0; i < d.arrays; ++i) take(&m->dz[i], dz);
    return true;
}
inline void release(const DenseMemory &m) {
    if (!m.base) return;
    int cur = -1;
    bool switched = false;
    if (own(hipGetDevice(&cur)) == hipSuccess && cur != m.device) switched = own(hipSetDevice(m.device)) == hipSuccess;
    // teardown is best effort: a failure here leaves nothing to undo
    (void)own(hipFree(m.base));
    if (switched) (void)own(hipSetDevice(cur));
}

// An operand whose rows can be loaded 16 bytes at a time without a look at
// their ends: `cols` long, ld apart.
inline bool direct_rows(const void *p, int64_t cols, int64_t ld) { return cols % 8 == 0 && ld % 8 == 0 && aligned(p, 16); }
// An output row on 16 bytes (of `elem` each).
inline bool wide_rows(const void *p, int64_t ld, int64_t elem) { return ld * elem % 16 == 0 && aligned(p, 16); }

// One or two arrays of an operand, or their padded copies.
struct DenseOperand {
    const uint16_t *p[2];
    int64_t ld;
    bool direct;
};
// `to`: room for copies, made by the launch of `pads`, or nulls.
constexpr uint16_t *kNoRoom[2] = {};
inline DenseOperand operand(const uint16_t *p0, const uint16_t *p1, int64_t rows, int64_t cols, int64_t ld, uint16_t *const *to, PadArgs *pads) {
    const int n = p1 ? 2 : 1;
    DenseOperand o = {{p0, p1 ? p1 : p0}, ld, direct_rows(p0, cols, ld) && aligned(p1, 16)};
    if (o.direct || !to[0] || (n > 1 && !to[1])) return o;
    for (int i = 0; i < n; ++i) {
        pads->m[pads->count++] = {o.p[i], to[i], rows, cols, ld, up8(cols)};
        o.p[i] = to[i];
    }
    if (n == 1) o.p[1] = o.p[0];
    o.ld = up8(cols);
    o.direct = true;
    return o;
}

// The forward product or pair: `a` holds what the epilogue needs.
template <TileKind KIND>
inline hipError_t dense_forward(DenseArgs &a, const DenseSizes &d, const DenseMemory &m, int64_t rows, const void *x, const void *w0,
                                const void *w1, hipStream_t s) {
    const bool kn = d.layout == GEMM_WEIGHTS_KN;
    PadArgs pads = {};
    const bool as_is = dense_as_it_is(rows, d.K, kn);
    const DenseOperand A = operand((const uint16_t *)x, nullptr, rows, d.K, d.ldx, as_is ? kNoRoom : &m.x, &pads);
    const DenseOperand B = operand((const uint16_t *)w0, (const uint16_t *)w1, kn ? d.K : d.N, kn ? d.N : d.K, d.ldw, as_is ? kNoRoom : m.w, &pads);
    a.rows = rows;
    a.N = d.N;
    a.K = d.K;
    a.lda = A.ld;
    a.ldb = B.ld;
    a.act = d.act;
    a.slots = m.slots;
    const bool direct = A.direct && B.direct;
    // (without both, what could be copied is used as it is)
    for (int i = 0; i < 2; ++i) {
        a.A[i] = direct ? A.p[i] : (const uint16_t *)x;
        a.B[i] = direct ? B.p[i] : (const uint16_t *)(i && w1 ? w1 : w0);
    }
    if (!direct) {
        a.lda = d.ldx;
        a.ldb = d.ldw;
    } else {
        const hipError_t e = launch_padded_copies(pads, s);
        if (e != hipSuccess) return e;
    }
    return launch_dense<KIND>(a, kn, direct, m.slot_bytes, s);
}

// Gradients of x and of the weights from dz (row stride d.ldd), which `copied` says
// lies in its padded copy already.
struct DenseBackward {
    int64_t rows;
    int32_t dw_f32, add;
    bool copied;
    const void *x, *w[2], *dz[2];     // the second ones null, but for a pair
    void *dx, *dw[2];
    int64_t lddx, lddw;
};
template <TileKind SUM>
inline hipError_t dense_backward(const DenseBackward &b, const DenseSizes &d, const DenseMemory &m, hipStream_t s) {
    const bool kn = d.layout == GEMM_WEIGHTS_KN, some = b.rows > 0;
    PadArgs pads = {};
    auto of = [](const void *p) { return (const uint16_t *)p; };
    const DenseOperand none = {{nullptr, nullptr}, 0, false};
    DenseOperand Z, W = none, X = none;
    if (b.copied) Z = {{m.dz[0], m.dz[1] ? m.dz[1] : m.dz[0]}, up8(d.N), true};
    else if (some && (b.dx || b.dw[0])) Z = operand(of(b.dz[0]), of(b.dz[1]), b.rows, d.N, d.ldd, m.dz, &pads);
    else Z = {{of(b.dz[0]), of(b.dz[1] ? b.dz[1] : b.dz[0])}, d.ldd, false};
    if (some && b.dx && Z.direct)
        W = operand(of(b.w[0]), of(b.w[1]), kn ? d.K : d.N, kn ? d.N : d.K, d.ldw, dense_as_it_is(b.rows, d.N, !kn) ? kNoRoom : m.w, &pads);
    if (some && b.dw[0] && Z.direct) X = operand(of(b.x), nullptr, b.rows, d.K, d.ldx, &m.x, &pads);
    hipError_t e = launch_padded_copies(pads, s);
    if (e != hipSuccess) return e;
    if (b.dx && some) {
        const bool direct = Z.direct && W.direct;
        DenseArgs a = {};
        a.rows = b.rows;
        a.N = d.K;
        a.K = d.N;
        a.lda = Z.ld;
        a.ldb = direct ? W.ld : d.ldw;
        for (int i = 0; i < 2; ++i) {
            a.A[i] = Z.p[i];
            a.B[i] = direct ? W.p[i] : of(i && b.w[1] ? b.w[1] : b.w[0]);
        }
        a.D[0] = b.dx;
        a.ldd = b.lddx;
        a.slots = m.slots;
        e = launch_dense<SUM>(a, !kn, direct, m.slot_bytes, s);
        if (e != hipSuccess) return e;
    }
    if (b.dw[0]) {
        const bool direct = Z.direct && X.direct;
        const uint16_t *const x = direct ? X.p[0] : of(b.x);
        const int64_t ldx = direct ? X.ld : d.ldx;
        DenseArgs a = {};
        a.rows = kn ? d.K : d.N;
        a.N = kn ? d.N : d.K;
        a.K = b.rows;
        a.count = d.arrays;
        for (int i = 0; i < 2; ++i) {
            a.A[i] = kn ? x : Z.p[i];
            a.B[i] = kn ? Z.p[i] : x;
            a.D[i] = b.dw[i];
        }
        a.lda = kn ? ldx : Z.ld;
        a.ldb = kn ? Z.ld : ldx;
        a.ldd = b.lddw;
        a.out_f32 = b.dw_f32;
        a.add = b.add;
        a.slots = m.slots;
        return launch_weight_gradients(a, direct, m.slot_bytes, s);
    }
    return hipSuccess;
}

}  // namespace ffn
}  // namespace gemm_rs
