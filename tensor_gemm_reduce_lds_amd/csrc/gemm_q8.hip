// 8-bit integer product with scales per token and channel (gemm_q8.h).
#include <stdlib.h>

#include "gemm_q8.h"
#include "mma_tile.h"

using namespace gemm_rs::ffn;

namespace {

constexpr int64_t kMaxK = int64_t(1) << 17;
constexpr int64_t kMaxStride = int64_t(1) << 23;

struct Q8Args {
    int64_t M, N, K, lda, ldw, ldd;
    const int8_t *a, *w;
    const float *a_scale, *w_scale, *bias;
    void *D;
    int32_t out_f32;
};

__device__ __forceinline__ void store_one(const Q8Args &p, int64_t m, int64_t n, int32_t acc) {
    float v = (float)acc * p.a_scale[m];
    v = p.bias ? __builtin_fmaf(v, p.w_scale[n], p.bias[n]) : v * p.w_scale[n];
    if (p.out_f32) ((float *)p.D)[m * p.ldd + n] = v;
    else ((uint16_t *)p.D)[m * p.ldd + n] = (uint16_t)to_bf16(v);
}

// 64 x 64 outputs per workgroup, 32 x 32 per wave, 128 bytes of the
// contraction at a time through LDS rows of 144 bytes.
__global__ __launch_bounds__(256) void q8_tile_kernel(Q8Args p) {
    constexpr int PITCH = 144;
    __shared__ __attribute__((aligned(16))) char As[64 * PITCH], Ws[64 * PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    i32x16_t acc = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += 128) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 32 + (tid >> 3), c = (tid & 7) * 16;
            const bool in = k0 + c < p.K;      // K is a multiple of 16
            i32x4_t av = {}, wv = {};
            if (in && m0 + r < p.M) av = *(const i32x4_t *)(p.a + (m0 + r) * p.lda + k0 + c);
            if (in && n0 + r < p.N) wv = *(const i32x4_t *)(p.w + (n0 + r) * p.ldw + k0 + c);
            *(i32x4_t *)(As + r * PITCH + c) = av;
            *(i32x4_t *)(Ws + r * PITCH + c) = wv;
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int c = s * 32 + (lane >> 5) * 16;
            acc = mma(*(const i32x4_t *)(As + (wm + (lane & 31)) * PITCH + c),
                      *(const i32x4_t *)(Ws + (wn + (lane & 31)) * PITCH + c), acc);
        }
        __syncthreads();
    }
    const int64_t m = m0 + wm + (lane & 31);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int64_t n = n0 + wn + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
        if (m < p.M && n < p.N) store_one(p, m, n, acc[v]);
    }
}

// One row per workgroup, read twice (the second time from the caches).
template <bool F32, int VEC>
__global__ __launch_bounds__(256) void quantize_kernel(const void *x, int64_t rows, int64_t cols,
                                                       int64_t ldx, int8_t *q, int64_t ldq,
                                                       float *scale) {
    __shared__ float slots[2 * 16];
    int turn = 0;
    const int64_t padded = (cols + 15) / 16 * 16;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        float m[1] = {0.0f};
        for (int64_t c = threadIdx.x * VEC; c < cols; c += 256 * VEC) {
            Raw<F32, VEC> r;
            load_raw(r, x, row * ldx + c);
#pragma unroll
            for (int e = 0; e < VEC; ++e) m[0] = MaxBits::join(m[0], fabsf(raw_at(r, e)));
        }
        block_join<MaxBits, 256, 1>(m, slots, turn);
        const QuantRow k = quant_row(m[0]);
        if (threadIdx.x == 0) scale[row] = k.scale;
        for (int64_t c = threadIdx.x * VEC; c < padded; c += 256 * VEC) {
            Raw<F32, VEC> r = {};
            if (c < cols) load_raw(r, x, row * ldx + c);
            int8_t *to = q + row * ldq + c;
            if constexpr (VEC == 8) {
                u32x2_t w = {0u, 0u};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e >> 2] |= (uint32_t)(quant_one(k, raw_at(r, e)) & 0xff) << (8 * (e & 3));
                *(u32x2_t *)to = w;
            } else {
                *to = (int8_t)quant_one(k, raw_at(r, 0));
            }
        }
    }
}

int validate(const gemm_q8_desc_t &d) {
    if (d.M < 1 || d.N < 1 || d.K < 1 || d.lda < 0 || d.ldw < 0 || d.ldd < 0)
        return GEMM_RS_ERR_INVALID_ARG;
    if (!known_type(d.out_dtype) || (d.has_bias != 0 && d.has_bias != 1))
        return GEMM_RS_ERR_INVALID_ARG;
    if ((d.lda && d.lda < d.K) || (d.ldw && d.ldw < d.K) || (d.ldd && d.ldd < d.N))
        return GEMM_RS_ERR_INVALID_ARG;
    if (d.K % 16 || d.lda % 16 || d.ldw % 16) return GEMM_RS_ERR_UNSUPPORTED;
    if (d.K >= kMaxK || d.M > INT32_MAX || d.N > INT32_MAX) return GEMM_RS_ERR_UNSUPPORTED;
    if (d.lda >= kMaxStride || d.ldw >= kMaxStride || d.ldd > INT32_MAX)
        return GEMM_RS_ERR_UNSUPPORTED;
    return GEMM_RS_OK;
}

}  // namespace

struct gemm_q8_plan_s {
    gemm_q8_desc_t d;    // strides filled in
    int device;
};

extern "C" {

int gemm_q8_plan(const gemm_q8_desc_t *desc, gemm_q8_plan_t *out) {
    if (!desc || !out) return GEMM_RS_ERR_INVALID_ARG;
    *out = nullptr;
    const int rc = validate(*desc);
    if (rc != GEMM_RS_OK) return rc;
    gemm_q8_plan_s *p = (gemm_q8_plan_s *)calloc(1, sizeof(gemm_q8_plan_s));
    if (!p) return GEMM_RS_ERR_HIP;
    p->d = *desc;
    if (!p->d.lda) p->d.lda = p->d.K;
    if (!p->d.ldw) p->d.ldw = p->d.K;
    if (!p->d.ldd) p->d.ldd = p->d.N;
    if (hipGetDevice(&p->device) != hipSuccess) {
        free(p);
        return GEMM_RS_ERR_HIP;
    }
    *out = p;
    return GEMM_RS_OK;
}

int gemm_q8_run(gemm_q8_plan_t p, const void *a, const void *a_scale, const void *w,
                const void *w_scale, const void *bias, void *D, int64_t rows, void *stream) {
    if (!p || !on_device(p->device)) return GEMM_RS_ERR_INVALID_ARG;
    const gemm_q8_desc_t &d = p->d;
    if (rows < 0 || rows > d.M) return GEMM_RS_ERR_INVALID_ARG;
    if (!a || !a_scale || !w || !w_scale || !D || (bias != nullptr) != (d.has_bias != 0))
        return GEMM_RS_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
        !aligned(bias, 4) || !aligned(D, type_bytes(d.out_dtype)))
        return GEMM_RS_ERR_INVALID_ARG;
    if (rows == 0) return GEMM_RS_OK;
    Q8Args q = {};
    q.M = rows;
    q.N = d.N;
    q.K = d.K;
    q.lda = d.lda;
    q.ldw = d.ldw;
    q.ldd = d.ldd;
    q.a = (const int8_t *)a;
    q.w = (const int8_t *)w;
    q.a_scale = (const float *)a_scale;
    q.w_scale = (const float *)w_scale;
    q.bias = (const float *)bias;
    q.D = D;
    q.out_f32 = d.out_dtype == GEMM_RS_F32;
    hipLaunchKernelGGL(q8_tile_kernel, dim3((unsigned)((d.N + 63) / 64), (unsigned)((rows + 63) / 64)),
                       dim3(256), 0, (hipStream_t)stream, q);
    return hipGetLastError() == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int gemm_q8_quantize(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, void *q,
                     int64_t ldq, void *scale, void *stream) {
    if (!known_type(dtype) || rows < 0 || cols < 1 || ldx < cols || ldq < (cols + 15) / 16 * 16)
        return GEMM_RS_ERR_INVALID_ARG;
    if (!x || !q || !scale || !aligned(x, type_bytes(dtype)) || !aligned(scale, 4))
        return GEMM_RS_ERR_INVALID_ARG;
    if (cols >= kMaxK || rows > INT32_MAX || ldx > INT32_MAX || ldq > INT32_MAX)
        return GEMM_RS_ERR_UNSUPPORTED;
    if (rows == 0) return GEMM_RS_OK;
    const bool vec = cols % 8 == 0 && ldx % 8 == 0 && ldq % 8 == 0 && aligned(x, 16) && aligned(q, 8);
    const dim3 grid((unsigned)(rows < 65536 ? rows : 65536));
    hipStream_t s = (hipStream_t)stream;
    auto go = [&](auto *kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, x, rows, cols, ldx, (int8_t *)q, ldq,
                           (float *)scale);
    };
    if (dtype == GEMM_RS_F32) vec ? go(quantize_kernel<true, 8>) : go(quantize_kernel<true, 1>);
    else vec ? go(quantize_kernel<false, 8>) : go(quantize_kernel<false, 1>);
    return hipGetLastError() == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int gemm_q8_query(gemm_q8_plan_t p, gemm_q8_info_t *info) {
    if (!p || !info) return GEMM_RS_ERR_INVALID_ARG;
    info->workspace_bytes = 0;
    return GEMM_RS_OK;
}

int gemm_q8_destroy(gemm_q8_plan_t p) {
    free(p);
    return GEMM_RS_OK;
}

}  // extern "C"
