// The matrix product with bias, activation and residual (gemm_epi.h).
#include "gemm_epi.h"
#include "dense_host.h"

using namespace gemm_rs::ffn;

namespace {

int validate(const gemm_epi_desc_t &d) {
    const DenseSizes z = {d.M, d.N, d.K, d.layout, d.act, 1, d.backward};
    const int rc = check_sizes(z);
    if (rc != GEMM_RS_OK) return rc;
    if (!flag(d.has_bias) || !flag(d.has_residual) || !flag(d.backward) || !flag(d.accumulate) || !known_type(d.out_dtype) ||
        !known_type(d.bias_dtype) || !known_type(d.z_dtype) || !known_type(d.dw_dtype))
        return GEMM_RS_ERR_INVALID_ARG;
    const int64_t wcols = d.layout == GEMM_WEIGHTS_KN ? d.N : d.K;
    if (!stride_ok(d.ldx, d.K) || !stride_ok(d.ldw, wcols) || !stride_ok(d.ldr, d.N) || !stride_ok(d.ldy, d.N) || !stride_ok(d.ldz, d.N) ||
        !stride_ok(d.lddy, d.N) || !stride_ok(d.lddz, d.N) || !stride_ok(d.lddx, d.K) || !stride_ok(d.lddw, wcols))
        return GEMM_RS_ERR_INVALID_ARG;
    const int64_t ld[] = {d.ldx, d.ldw, d.ldr, d.ldy, d.ldz, d.lddy, d.lddz, d.lddx, d.lddw};
    return check_limits(z, ld, 9);
}

// dz is not dy itself
bool through(const gemm_epi_desc_t &d) { return d.act != GEMM_ACT_NONE || d.out_dtype == GEMM_RS_F32; }

}  // namespace

struct gemm_epi_plan_s {
    gemm_epi_desc_t d;        // strides filled in
    DenseSizes size;
    DenseMemory mem;
};

extern "C" {

int gemm_epi_plan(const gemm_epi_desc_t *desc, gemm_epi_plan_t *out) {
    if (!desc || !out) return GEMM_RS_ERR_INVALID_ARG;
    *out = nullptr;
    const int rc = validate(*desc);
    if (rc != GEMM_RS_OK) return rc;
    gemm_epi_plan_s *p = (gemm_epi_plan_s *)calloc(1, sizeof(gemm_epi_plan_s));
    if (!p) return GEMM_RS_ERR_HIP;
    gemm_epi_desc_t &d = p->d;
    d = *desc;
    const int64_t wcols = d.layout == GEMM_WEIGHTS_KN ? d.N : d.K;
    for (int64_t *ld : {&d.ldr, &d.ldy, &d.ldz, &d.lddy, &d.lddz})
        if (!*ld) *ld = d.N;
    for (int64_t *ld : {&d.ldx, &d.lddx})
        if (!*ld) *ld = d.K;
    for (int64_t *ld : {&d.ldw, &d.lddw})
        if (!*ld) *ld = wcols;
    p->size = {d.M, d.N, d.K, d.layout, d.act, 1, d.backward, d.has_bias, d.dw_dtype == GEMM_RS_F32, d.ldx, d.ldw, through(d) ? d.lddz : d.lddy};
    if (!allocate(&p->mem, p->size)) {
        release(p->mem);
        free(p);
        return GEMM_RS_ERR_HIP;
    }
    *out = p;
    return GEMM_RS_OK;
}

int gemm_epi_run(gemm_epi_plan_t p, const void *x, const void *w, const void *bias, const void *r, void *y, void *z, int64_t rows,
                 void *stream) {
    if (!p || !on_device(p->mem.device)) return GEMM_RS_ERR_INVALID_ARG;
    const gemm_epi_desc_t &d = p->d;
    if (rows < 0 || rows > d.M) return GEMM_RS_ERR_INVALID_ARG;
    const size_t oe = type_bytes(d.out_dtype), ze = type_bytes(d.z_dtype);
    const bool some = rows > 0;
    if (!w || !bias == !!d.has_bias || (r && !d.has_residual) || (some && (!x || !y || (d.has_residual && !r))))
        return GEMM_RS_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(w, 2) || !aligned(bias, type_bytes(d.bias_dtype)) || !aligned(r, oe) || !aligned(y, oe) || !aligned(z, ze))
        return GEMM_RS_ERR_INVALID_ARG;
    if (!in_place_ok(y, r, true, rows, d.ldy, d.ldr)) return GEMM_RS_ERR_INVALID_ARG;
    if (!some) return GEMM_RS_OK;
    DenseArgs a = {};
    a.bias_f32 = d.bias_dtype == GEMM_RS_F32;
    a.bias[0] = bias;
    a.out_f32 = d.out_dtype == GEMM_RS_F32;
    a.R = r;
    a.ldr = d.ldr;
    a.D[0] = y;
    a.ldd = d.ldy;
    a.Z[0] = z;
    a.z_f32 = d.z_dtype == GEMM_RS_F32;
    a.ldz = d.ldz;
    return dense_forward<kOne>(a, p->size, p->mem, rows, x, w, nullptr, (hipStream_t)stream) == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int gemm_epi_backward(gemm_epi_plan_t p, const void *dy, const void *x, const void *w, const void *z, void *dz, void *dx, void *dw,
                      void *dbias, int64_t rows, void *stream) {
    if (!p || !on_device(p->mem.device)) return GEMM_RS_ERR_INVALID_ARG;
    const gemm_epi_desc_t &d = p->d;
    if (!d.backward || rows < 0 || rows > d.M) return GEMM_RS_ERR_INVALID_ARG;
    const bool f32 = d.out_dtype == GEMM_RS_F32, own_dz = through(d);
    const int64_t ye = f32 ? 4 : 2, ze = (int64_t)type_bytes(d.z_dtype);
    const bool some = rows > 0;
    if ((dbias && !d.has_bias) || (z && d.act == GEMM_ACT_NONE) || (dz && !own_dz)) return GEMM_RS_ERR_INVALID_ARG;
    if (some && (!dy || (d.act != GEMM_ACT_NONE && !z) || (own_dz && !dz) || (dw && !x) || (dx && !w))) return GEMM_RS_ERR_INVALID_ARG;
    if (!aligned(dy, ye) || !aligned(x, 2) || !aligned(w, 2) || !aligned(z, ze) || !aligned(dz, 2) || !aligned(dx, 2) ||
        !aligned(dw, type_bytes(d.dw_dtype)) || !aligned(dbias, 4))
        return GEMM_RS_ERR_INVALID_ARG;
    if (!in_place_ok(dz, z, ze == 2, rows, d.lddz, d.ldz) || !in_place_ok(dz, dy, !f32, rows, d.lddz, d.lddy)) return GEMM_RS_ERR_INVALID_ARG;
    if (!some && d.accumulate) return GEMM_RS_OK;
    hipStream_t s = (hipStream_t)stream;
    // dz into a padded copy too, where one is needed and has room
    const bool copied = some && own_dz && p->mem.dz[0] && (dx || dw);
    if ((some && own_dz) || dbias) {
        ActGradArgs a = {};
        a.rows = rows;
        a.N = d.N;
        a.act = d.act;
        a.dy_f32 = f32;
        a.add = d.accumulate;
        a.dy = dy;
        a.Z[0] = z;
        a.z_f32 = d.z_dtype == GEMM_RS_F32;
        a.dZ[0] = (uint16_t *)dz;
        a.copy[0] = copied ? p->mem.dz[0] : nullptr;
        a.copy_ld = up8(d.N);
        a.db[0] = (float *)dbias;
        a.ldy = d.lddy;
        a.ldz = d.ldz;
        a.lddz = d.lddz;
        a.sums = p->mem.slots;
        a.wide = d.N % 8 == 0 && wide_rows(dy, d.lddy, ye) && (!z || wide_rows(z, d.ldz, ze)) && (!dz || wide_rows(dz, d.lddz, 2));
        if (launch_activation_gradient(a, p->mem.slot_bytes, s) != hipSuccess) return GEMM_RS_ERR_HIP;
    }
    DenseBackward b = {};
    b.rows = rows;
    b.dw_f32 = d.dw_dtype == GEMM_RS_F32;
    b.add = d.accumulate;
    b.copied = copied;
    b.x = x;
    b.w[0] = w;
    b.dz[0] = own_dz ? dz : dy;
    b.dx = dx;
    b.dw[0] = dw;
    b.lddx = d.lddx;
    b.lddw = d.lddw;
    return dense_backward<kOne>(b, p->size, p->mem, s) == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int gemm_epi_query(gemm_epi_plan_t p, gemm_epi_info_t *info) {
    if (!p || !info) return GEMM_RS_ERR_INVALID_ARG;
    info->workspace_bytes = p->mem.bytes;
    return GEMM_RS_OK;
}

int gemm_epi_destroy(gemm_epi_plan_t p) {
    if (!p) return GEMM_RS_OK;
    release(p->mem);
    free(p);
    return GEMM_RS_OK;
}

}  // extern "C"
