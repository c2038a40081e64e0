// The gated projections of a feed-forward block (gemm_gated.h).
#include "gemm_gated.h"
#include "dense_host.h"

using namespace gemm_rs::ffn;

namespace {

int validate(const gemm_gated_desc_t &d) {
    const DenseSizes z = {d.M, d.N, d.K, d.layout, d.act, 2, d.backward};
    const int rc = check_sizes(z);
    if (rc != GEMM_RS_OK) return rc;
    if (!flag(d.has_bias) || !flag(d.backward) || !flag(d.accumulate) || !known_type(d.bias_dtype) || !known_type(d.z_dtype) ||
        !known_type(d.dw_dtype))
        return GEMM_RS_ERR_INVALID_ARG;
    const int64_t wcols = d.layout == GEMM_WEIGHTS_KN ? d.N : d.K;
    if (!stride_ok(d.ldx, d.K) || !stride_ok(d.ldw, wcols) || !stride_ok(d.ldh, d.N) || !stride_ok(d.ldz, d.N) || !stride_ok(d.lddh, d.N) ||
        !stride_ok(d.lddz, d.N) || !stride_ok(d.lddx, d.K) || !stride_ok(d.lddw, wcols))
        return GEMM_RS_ERR_INVALID_ARG;
    const int64_t ld[] = {d.ldx, d.ldw, d.ldh, d.ldz, d.lddh, d.lddz, d.lddx, d.lddw};
    return check_limits(z, ld, 8);
}

}  // namespace

struct gemm_gated_plan_s {
    gemm_gated_desc_t d;      // strides filled in
    DenseSizes size;
    DenseMemory mem;
};

extern "C" {

int gemm_gated_plan(const gemm_gated_desc_t *desc, gemm_gated_plan_t *out) {
    if (!desc || !out) return GEMM_RS_ERR_INVALID_ARG;
    *out = nullptr;
    const int rc = validate(*desc);
    if (rc != GEMM_RS_OK) return rc;
    gemm_gated_plan_s *p = (gemm_gated_plan_s *)calloc(1, sizeof(gemm_gated_plan_s));
    if (!p) return GEMM_RS_ERR_HIP;
    gemm_gated_desc_t &d = p->d;
    d = *desc;
    const int64_t wcols = d.layout == GEMM_WEIGHTS_KN ? d.N : d.K;
    for (int64_t *ld : {&d.ldh, &d.ldz, &d.lddh, &d.lddz})
        if (!*ld) *ld = d.N;
    for (int64_t *ld : {&d.ldx, &d.lddx})
        if (!*ld) *ld = d.K;
    for (int64_t *ld : {&d.ldw, &d.lddw})
        if (!*ld) *ld = wcols;
    p->size = {d.M, d.N, d.K, d.layout, d.act, 2, d.backward, d.has_bias, d.dw_dtype == GEMM_RS_F32, d.ldx, d.ldw, d.lddz};
    if (!allocate(&p->mem, p->size)) {
        release(p->mem);
        free(p);
        return GEMM_RS_ERR_HIP;
    }
    *out = p;
    return GEMM_RS_OK;
}

int gemm_gated_run(gemm_gated_plan_t p, const void *x, const void *w_gate, const void *w_up, const void *b_gate, const void *b_up, void *h,
                   void *z_gate, void *z_up, int64_t rows, void *stream) {
    if (!p || !on_device(p->mem.device)) return GEMM_RS_ERR_INVALID_ARG;
    const gemm_gated_desc_t &d = p->d;
    if (rows < 0 || rows > d.M) return GEMM_RS_ERR_INVALID_ARG;
    const size_t be = type_bytes(d.bias_dtype), ze = type_bytes(d.z_dtype);
    const bool some = rows > 0;
    if ((!x && some) || !w_gate || !w_up || !b_gate == !!d.has_bias || !b_up == !!d.has_bias || !z_gate != !z_up ||
        (some && !h && !z_gate))
        return GEMM_RS_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(w_gate, 2) || !aligned(w_up, 2) || !aligned(b_gate, be) || !aligned(b_up, be) || !aligned(h, 2) ||
        !aligned(z_gate, ze) || !aligned(z_up, ze))
        return GEMM_RS_ERR_INVALID_ARG;
    if (!some) return GEMM_RS_OK;
    DenseArgs a = {};
    a.bias_f32 = d.bias_dtype == GEMM_RS_F32;
    a.bias[0] = b_gate;
    a.bias[1] = b_up;
    a.D[0] = h;
    a.ldd = d.ldh;
    a.Z[0] = z_gate;
    a.Z[1] = z_up;
    a.z_f32 = d.z_dtype == GEMM_RS_F32;
    a.ldz = d.ldz;
    return dense_forward<kPair>(a, p->size, p->mem, rows, x, w_gate, w_up, (hipStream_t)stream) == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int gemm_gated_backward(gemm_gated_plan_t p, const void *dh, const void *x, const void *w_gate, const void *w_up, const void *z_gate,
                        const void *z_up, void *dz_gate, void *dz_up, void *dx, void *dw_gate, void *dw_up, void *db_gate, void *db_up,
                        int64_t rows, void *stream) {
    if (!p || !on_device(p->mem.device)) return GEMM_RS_ERR_INVALID_ARG;
    const gemm_gated_desc_t &d = p->d;
    if (!d.backward || rows < 0 || rows > d.M) return GEMM_RS_ERR_INVALID_ARG;
    const size_t we = type_bytes(d.dw_dtype), ze = type_bytes(d.z_dtype);
    const bool some = rows > 0;
    if (!dw_gate != !dw_up || !db_gate != !db_up || (db_gate && !d.has_bias)) return GEMM_RS_ERR_INVALID_ARG;
    if (some && (!dh || !z_gate || !z_up || !dz_gate || !dz_up || (dw_gate && !x) || (dx && (!w_gate || !w_up)))) return GEMM_RS_ERR_INVALID_ARG;
    for (const void *q : {dh, x, w_gate, w_up, (const void *)dz_gate, (const void *)dz_up, (const void *)dx})
        if (!aligned(q, 2)) return GEMM_RS_ERR_INVALID_ARG;
    if (!aligned(z_gate, ze) || !aligned(z_up, ze) || !aligned(dw_gate, we) || !aligned(dw_up, we) || !aligned(db_gate, 4) || !aligned(db_up, 4)) return GEMM_RS_ERR_INVALID_ARG;
    for (const void *out : {dz_gate, dz_up})
        for (const void *in : {z_gate, z_up})
            if (!in_place_ok(out, in, ze == 2, rows, d.lddz, d.ldz)) return GEMM_RS_ERR_INVALID_ARG;
    if (!some && d.accumulate) return GEMM_RS_OK;
    hipStream_t s = (hipStream_t)stream;
    // dz into a padded copy too, where one is needed and has room
    const bool copied = some && p->mem.dz[0] && (dx || dw_gate);
    if (some || db_gate) {
        ActGradArgs a = {};
        a.rows = rows;
        a.N = d.N;
        a.act = d.act;
        a.pair = 1;
        a.add = d.accumulate;
        a.dy = dh;
        a.Z[0] = z_gate;
        a.Z[1] = z_up;
        a.z_f32 = d.z_dtype == GEMM_RS_F32;
        a.dZ[0] = (uint16_t *)dz_gate;
        a.dZ[1] = (uint16_t *)dz_up;
        for (int i = 0; i < 2; ++i) a.copy[i] = copied ? p->mem.dz[i] : nullptr;
        a.copy_ld = up8(d.N);
        a.db[0] = (float *)db_gate;
        a.db[1] = (float *)db_up;
        a.ldy = d.lddh;
        a.ldz = d.ldz;
        a.lddz = d.lddz;
        a.sums = p->mem.slots;
        a.wide = d.N % 8 == 0 && wide_rows(dh, d.lddh, 2) && wide_rows(z_gate, d.ldz, (int64_t)ze) && aligned(z_up, 16) &&
                 wide_rows(dz_gate, d.lddz, 2) && aligned(dz_up, 16);
        if (launch_activation_gradient(a, p->mem.slot_bytes, s) != hipSuccess) return GEMM_RS_ERR_HIP;
    }
    DenseBackward b = {};
    b.rows = rows;
    b.dw_f32 = d.dw_dtype == GEMM_RS_F32;
    b.add = d.accumulate;
    b.copied = copied;
    b.x = x;
    b.w[0] = w_gate;
    b.w[1] = w_up;
    b.dz[0] = dz_gate;
    b.dz[1] = dz_up;
    b.dx = dx;
    b.dw[0] = dw_gate;
    b.dw[1] = dw_up;
    b.lddx = d.lddx;
    b.lddw = d.lddw;
    return dense_backward<kParts>(b, p->size, p->mem, s) == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int gemm_gated_query(gemm_gated_plan_t p, gemm_gated_info_t *info) {
    if (!p || !info) return GEMM_RS_ERR_INVALID_ARG;
    info->workspace_bytes = p->mem.bytes;
    return GEMM_RS_OK;
}

int gemm_gated_destroy(gemm_gated_plan_t p) {
    if (!p) return GEMM_RS_OK;
    release(p->mem);
    free(p);
    return GEMM_RS_OK;
}

}  // extern "C"
