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
    int32_t wide_out;     // rows of D can be stored 8 elements at a time
};

// float(acc) * a_scale, then * w_scale (+ bias, fused)
__device__ __forceinline__ float scaled(int32_t acc, float sa, float sw, const float *bias) {
    const float v = (float)acc * sa;
    return bias ? __builtin_fmaf(v, sw, *bias) : v * sw;
}

__device__ __forceinline__ void store_one(const Q8Args &p, int64_t m, int64_t n, float v) {
    if (p.out_f32) ((float *)p.D)[m * p.ldd + n] = v;
    else ((uint16_t *)p.D)[m * p.ldd + n] = (uint16_t)to_bf16(v);
}

// BM x BN outputs per workgroup.  An XCD gets a run of the tiles in groups of 8
// tile-rows, a group column by column.
template <int BM, int BN, int WGM, int WGN, int STAGES>
__global__ __launch_bounds__(64 * WGM * WGN) void q8_tile_kernel(Q8Args p) {
    using T = Tile<i32x16_t, BM, BN, WGM, WGN, false, false, STAGES>;
    extern __shared__ __attribute__((aligned(1024))) char smem_generic[];
    lds_t *smem = (lds_t *)smem_generic;
    const uint32_t tn = (uint32_t)((p.N + BN - 1) / BN), tm = (uint32_t)((p.M + BM - 1) / BM);
    const uint32_t t = xcd_run(blockIdx.x, tm * tn);
    const uint32_t g = t / (8 * tn), in = t - g * 8 * tn, rows = tm - g * 8 < 8 ? tm - g * 8 : 8;
    const int64_t m0 = (int64_t)(g * 8 + in % rows) * BM, n0 = (int64_t)(in / rows) * BN;
    const int32_t m_left = (int32_t)(p.M - m0 < BM ? p.M - m0 : BM);
    const int32_t n_left = (int32_t)(p.N - n0 < BN ? p.N - n0 : BN);
    T tile;
    const Operand a = {(const char *)p.a + m0 * p.lda, p.lda, m_left};
    const Operand w = {(const char *)p.w + n0 * p.ldw, p.ldw, n_left};
    tile.template run<1>(smem, a, w, (int32_t)p.K);
    // a lane's 8 columns are the same in every row it stores
    const int c0 = (int)(threadIdx.x % (BN / 8)) * 8;
    float sw[8], bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int64_t n = n0 + (c0 + e < n_left ? c0 + e : n_left - 1);
        sw[e] = p.w_scale[n];
        bias[e] = p.bias ? p.bias[n] : 0.0f;
    }
    tile.store(smem, [&](int r, int c, const int (&v)[8]) {
        if (r >= m_left || c >= n_left) return;
        const int64_t m = m0 + r;
        const float sa = p.a_scale[m];
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = scaled(v[e], sa, sw[e], p.bias ? &bias[e] : nullptr);
        if (p.wide_out && c + 8 <= n_left) {
            if (p.out_f32) store_vec<true, 8>(p.D, m * p.ldd + n0 + c, x);
            else store_vec<false, 8>(p.D, m * p.ldd + n0 + c, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < n_left) store_one(p, m, n0 + c + e, x[e]);
        }
    });
}

// Few rows: 16 channels and up to MB * 16 rows per workgroup, the contraction
// split over its 8 waves.  Every byte of w is used by one wave only, so
// operands go straight to registers, 64 bytes of each row per matrix
// operation; the waves' sums (integers: exact in any order) meet in LDS.
template <int MB>
__global__ __launch_bounds__(512) void q8_rows_kernel(Q8Args p) {
    constexpr int NW = 8, U = MB <= 2 ? 8 : 4;      // steps whose loads are in flight together
    __shared__ __attribute__((aligned(16))) int32_t part[NW][MB * 16][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int r = lane & 15, chunk = (lane >> 4) * 16;
    const int64_t n = n0 + r < p.N ? n0 + r : p.N - 1;
    const int8_t *wp = p.w + n * p.ldw + chunk;
    const int8_t *ap[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t m = b * 16 + r < p.M ? b * 16 + r : p.M - 1;
        ap[b] = p.a + m * p.lda + chunk;
    }
    const int K = (int)p.K, steps = (K + 63) / 64, per = (steps + NW - 1) / NW;
    const int s0 = wave * per;
    const int s1 = s0 + per < steps ? s0 + per : steps;
    i32x4_t acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = i32x4_t{0, 0, 0, 0};
    for (int s = s0; s < s1; s += U) {
        i32x4_t wf[U], af[U][MB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * 64;
            // the last step's chunks past K, and steps past this wave's, are 0
            const bool in = s + u < s1 && k + chunk < K;
            wf[u] = i32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int b = 0; b < MB; ++b) af[u][b] = i32x4_t{0, 0, 0, 0};
            if (in) {
                wf[u] = *(const i32x4_t *)(wp + k);
#pragma unroll
                for (int b = 0; b < MB; ++b) af[u][b] = *(const i32x4_t *)(ap[b] + k);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < MB; ++b) acc[b] = mma16(af[u][b], wf[u], acc[b]);
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) *(i32x4_t *)&part[wave][b * 16 + r][(lane >> 4) * 4] = acc[b];
    __syncthreads();
    for (int i = tid; i < MB * 256; i += 512) {
        const int64_t m = i >> 4, col = n0 + (i & 15);
        int32_t v = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += part[w][i >> 4][i & 15];
        if (m < p.M && col < p.N)
            store_one(p, m, col, scaled(v, p.a_scale[m], p.w_scale[col], p.bias ? p.bias + col : nullptr));
    }
}

// Rows of up to EPT * THREADS columns, one per workgroup, in registers; EPT
// 0: rows of any length, read twice (the second time from the caches).
template <bool F32, int VEC, int EPT, int THREADS>
__global__ __launch_bounds__(THREADS) void quantize_kernel(const void *x, int64_t rows, int64_t cols,
                                                           int64_t ldx, int8_t *q, int64_t ldq,
                                                           float *scale) {
    __shared__ float slots[2 * 16];
    int turn = 0;
    const int64_t padded = (cols + 15) / 16 * 16;
    constexpr int VPT = EPT ? EPT / VEC : 1;
    const int64_t t0 = (int64_t)threadIdx.x * VEC;
    auto put = [&](const QuantRow &k, const Raw<F32, VEC> &r, int8_t *to) {
        if constexpr (VEC == 8) {
            u32x2_t w = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e >> 2] |= (uint32_t)(quant_one(k, raw_at(r, e)) & 0xff) << (8 * (e & 3));
            *(u32x2_t *)to = w;
        } else {
            *to = (int8_t)quant_one(k, raw_at(r, 0));
        }
    };
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        Raw<F32, VEC> held[VPT];
        float m[1] = {0.0f};
        auto take = [&](Raw<F32, VEC> &r, int64_t c) {
            r = Raw<F32, VEC>{};
            if (c < cols) load_raw(r, x, row * ldx + c);
        };
        auto look = [&](const Raw<F32, VEC> &r) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) m[0] = MaxBits::join(m[0], fabsf(raw_at(r, e)));
        };
        if constexpr (EPT) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) take(held[k], t0 + k * THREADS * VEC);
#pragma unroll
            for (int k = 0; k < VPT; ++k) look(held[k]);
        } else {
            for (int64_t c = t0; c < cols; c += THREADS * VEC) {
                take(held[0], c);
                look(held[0]);
            }
        }
        block_join<MaxBits, THREADS, 1>(m, slots, turn);
        const QuantRow k = quant_row(m[0]);
        if (threadIdx.x == 0) scale[row] = k.scale;
        int8_t *const to = q + row * ldq;
        if constexpr (EPT) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t c = t0 + i * THREADS * VEC;
                if (c < padded) put(k, held[i], to + c);
            }
        } else {
            for (int64_t c = t0; c < padded; c += THREADS * VEC) {
                take(held[0], c);
                put(k, held[0], to + c);
            }
        }
    }
}

template <int BM, int BN, int WGM, int WGN, int STAGES>
hipError_t launch_tile(const Q8Args &q, hipStream_t s) {
    using T = Tile<i32x16_t, BM, BN, WGM, WGN, false, false, STAGES>;
    return launch_lds<q8_tile_kernel<BM, BN, WGM, WGN, STAGES>>(
        ((q.M + BM - 1) / BM) * ((q.N + BN - 1) / BN), T::THREADS, T::LDS_BYTES, s, q);
}

hipError_t launch_product(const Q8Args &q, hipStream_t s) {
    if (q.M <= 128) {
        auto go = [&](auto *kernel) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)((q.N + 15) / 16)), dim3(512), 0, s, q);
            return hipGetLastError();
        };
        if (q.M <= 16) return go(q8_rows_kernel<1>);
        if (q.M <= 32) return go(q8_rows_kernel<2>);
        if (q.M <= 64) return go(q8_rows_kernel<4>);
        return go(q8_rows_kernel<8>);
    }
    const int64_t big = ((q.M + 255) / 256) * ((q.N + 255) / 256);
    if (big >= kCus * 3 / 4) return launch_tile<256, 256, 2, 4, 2>(q, s);
    return launch_tile<128, 128, 2, 2, 4>(q, s);
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
    q.wide_out = d.ldd % 8 == 0 && aligned(D, 16);
    return launch_product(q, (hipStream_t)stream) == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
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
    auto go = [&](auto *kernel, int threads) {
        hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, (hipStream_t)stream, x, rows, cols, ldx,
                           (int8_t *)q, ldq, (float *)scale);
    };
    auto of_type = [&](auto f32) {
        constexpr bool F = decltype(f32)::value;
        if (!vec) go(quantize_kernel<F, 1, 0, 256>, 256);
        else if (cols <= 2048) go(quantize_kernel<F, 8, 8, 256>, 256);
        else if (cols <= 8192) go(quantize_kernel<F, 8, 16, 512>, 512);
        else if (cols <= 16384) go(quantize_kernel<F, 8, 16, 1024>, 1024);
        else go(quantize_kernel<F, 8, 0, 256>, 256);
    };
    if (dtype == GEMM_RS_F32) of_type(std::true_type{});
    else of_type(std::false_type{});
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
