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

// A tile's sums from row m0 and column n0 on, scaled and stored.  A lane's columns
// are the same in every row it stores.
template <bool F32, class T>
__device__ __forceinline__ void store_tile(const Q8Args &p, const T &tile, lds_t *smem, int64_t m0, int32_t m_left, int64_t n0,
                                           int32_t n_left) {
    const int lane = (int)(threadIdx.x % (T::BN / 8));
    const int from[2] = {F32 ? lane * 4 : lane * 8, F32 ? lane * 4 + T::BN / 2 : lane * 8 + 4};
    float sw[8], bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int64_t c = n0 + from[e / 4] + e % 4, n = c < p.N ? c : p.N - 1;
        sw[e] = p.w_scale[n];
        bias[e] = p.bias ? p.bias[n] : 0.0f;
    }
    const uint32_t cols = (uint32_t)p.N;
    tile.template store<F32>(smem, [&](int r, int c, int d, const int (&v)[8]) {
        if (r >= m_left || c >= n_left) return;
        const int64_t m = m0 + r;
        const float sa = p.a_scale[m];
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = scaled(v[e], sa, sw[e], p.bias ? &bias[e] : nullptr);
        void *const to = row_of(p.D, m, p.ldd, F32 ? 4 : 2);
        const uint32_t at = (uint32_t)(n0 + c), next = (uint32_t)(n0 + d);
        if constexpr (F32) {
            if (p.wide_out) store4<true>((float *)to, at, cols, x);
            else store4<false>((float *)to, at, cols, x);
            if (d >= n_left) return;
            if (p.wide_out) store4<true>((float *)to, next, cols, x + 4);
            else store4<false>((float *)to, next, cols, x + 4);
        } else {
            if (p.wide_out) store8<false, true>(to, at, cols, x);
            else store8<false, false>(to, at, cols, x);
        }
    });
}

// BM x BN outputs per workgroup.  An XCD gets a run of the tiles in groups of 8
// tile-rows, a group column by column.  8192 x 8192 x 3584: 236 us, 2040 TOP/s (a
// library product of 8192^3 on the same card runs at 2260), at the board's power
// limit.  Rows of D that are not aligned are stored by the same 16-byte stores at
// any address (7174 x 1095 x 256: 15.5 us, one element per lane 20.4).
template <int BM, int BN, int WGM, int WGN, int SA, int SB>
__global__ __launch_bounds__(64 * WGM * WGN) void q8_tile_kernel(Q8Args p) {
    using T = Tile<i32x16_t, BM, BN, WGM, WGN, false, false, SA, SB>;
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
    if (p.out_f32) store_tile<true>(p, tile, smem, m0, m_left, n0, n_left);
    else store_tile<false>(p, tile, smem, m0, m_left, n0, n_left);
}

// Few rows: NB * 16 channels and up to MB * 16 rows per workgroup.  The
// contraction is dealt out to the NW waves 128 bytes at a time, and each wave
// streams its share through S stages of LDS of its own, so no wave waits for
// another until their sums (integers: exact in any order) meet at the end.
// Bound by reading w, and by the latency of launch, first loads and join where
// w is small: 1 x 8192 x 3584 7.4 us, 4.0 TB/s; 64 x 3584 x 8192 11 us, 2.7 TB/s
// (each stage also loads 64 rows of a, four times w's share).
template <int MB, int NB, int NW, int S>
struct RowsKernel {
    static constexpr int LOADS = (MB + NB) * 2;          // of 1 KB (8 rows) per stage
    static constexpr int STAGE = LOADS * 1024;
    static constexpr int LDS_BYTES = NW * S * STAGE;
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
    static_assert(MB * NB * 256 * 4 <= S * STAGE, "a wave's sums fit its stages");
    static_assert((S - 1) * LOADS < 64, "the load counter");

    static __device__ __forceinline__ int swz(int m) { return (m ^ (m >> 3)) & 7; }

    static __device__ void run(const Q8Args &p, lds_t *smem) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int n0 = blockIdx.x * NB * 16;
        const int n_left = (int)p.N - n0 < NB * 16 ? (int)p.N - n0 : NB * 16;
        const int K = (int)p.K, pieces = (K + 127) / 128;
        const int mine = pieces > wave ? (pieces - wave + NW - 1) / NW : 0;
        lds_t *const own = smem + wave * (S * STAGE);
        const uint32_t own_base = (uint32_t)(size_t)own;
        const uint32_t a_rows = (uint32_t)(p.M - 1) * (uint32_t)p.lda;      // bytes to the last row
        const uint32_t w_rows = (uint32_t)(n_left - 1) * (uint32_t)p.ldw;
        const char *const A = (const char *)p.a, *const W = (const char *)p.w + (int64_t)n0 * p.ldw;
        // rows past the last lie past the descriptors and read as zero
        uint32_t voff[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = (i < 2 * MB ? i : i - 2 * MB) * 8 + lane / 8;
            voff[i] = (uint32_t)r * (uint32_t)(i < 2 * MB ? p.lda : p.ldw) + (((lane & 7) ^ swz(r)) << 4);
        }
        auto issue = [&](int piece, int st) __attribute__((always_inline)) {
            const int k = (piece * NW + wave) * 128;
            const int left = K - k < 128 ? K - k : 128;
            const i32x4_t ra = buffer_of(A + k, a_rows + left), rw = buffer_of(W + k, w_rows + left);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                uint32_t v = voff[i];
                if (left < 128) {                       // chunks past K read as zero too
                    const int r = (i < 2 * MB ? i : i - 2 * MB) * 8 + lane / 8;
                    if ((((lane & 7) ^ swz(r)) << 4) >= left) v = 0xfffffff0u;
                }
                load_to_lds(i < 2 * MB ? ra : rw, v, own_base + st * STAGE + i * 1024);
            }
        };
        typedef __attribute__((address_space(3))) i32x4_t lds_i32x4;
        typedef __attribute__((address_space(3))) int32_t lds_i32;
        i32x4_t acc[MB][NB];
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int c = 0; c < NB; ++c) acc[b][c] = i32x4_t{0, 0, 0, 0};
        const int fr = lane & 15;       // fragments: row lane % 16, chunk 4 s + lane / 16
#pragma unroll
        for (int s = 0; s < S - 1; ++s)
            if (s < mine) issue(s, s);
        int st = 0;
        for (int i = 0; i < mine; ++i) {
            wait_groups<LOADS, S - 2>(mine - 1 - i);
            if (i + S - 1 < mine) issue(i + S - 1, st == 0 ? S - 1 : st - 1);
            i32x4_t af[2][MB], wf[2][NB];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int b = 0; b < MB; ++b)
                    af[s][b] = *(lds_i32x4 *)(own + st * STAGE + (b * 16 + fr) * 128 +
                                              (((4 * s + (lane >> 4)) ^ swz(b * 16 + fr)) << 4));
#pragma unroll
                for (int c = 0; c < NB; ++c)
                    wf[s][c] = *(lds_i32x4 *)(own + st * STAGE + (MB * 16 + c * 16 + fr) * 128 +
                                              (((4 * s + (lane >> 4)) ^ swz(c * 16 + fr)) << 4));
            }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int c = 0; c < NB; ++c) acc[b][c] = mma16(af[s][b], wf[s][c], acc[b][c]);
            // the reads are done before the next issue overwrites their stage
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (++st == S) st = 0;
        }
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int c = 0; c < NB; ++c)
                *(lds_i32x4 *)(own + ((b * 16 + fr) * (NB * 16) + c * 16 + (lane >> 4) * 4) * 4) = acc[b][c];
        __syncthreads();
        for (int i = tid; i < MB * NB * 256; i += NW * 64) {
            const int64_t m = i / (NB * 16), n = n0 + i % (NB * 16);
            int32_t v = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) v += *(lds_i32 *)(smem + w * (S * STAGE) + i * 4);
            if (m < p.M && n < p.N)
                store_one(p, m, n, scaled(v, p.a_scale[m], p.w_scale[n], p.bias ? p.bias + n : nullptr));
        }
    }
};

template <int MB, int NB, int NW, int S>
__global__ __launch_bounds__(NW * 64) void q8_rows_kernel(Q8Args p) {
    extern __shared__ __attribute__((aligned(1024))) char smem_generic[];
    RowsKernel<MB, NB, NW, S>::run(p, (lds_t *)smem_generic);
}

// q = rint(x * 127 * (1 / max|x|)), max / 127 beside it.  Rows of up to EPT *
// THREADS columns, one per workgroup, in registers; EPT 0: rows of any length,
// read twice (the second time from the caches).  Bound by memory: 8192 x 3584
// bf16 23 us, 3.8 TB/s; one row 2.2 us.
template <bool F32, bool WIDE, int EPT, int THREADS>
__global__ __launch_bounds__(THREADS) void quantize_kernel(const void *x, int64_t rows, uint32_t cols,
                                                           int64_t ldx, int8_t *q, int64_t ldq,
                                                           float *scale) {
    __shared__ JoinSlots<1> slots;
    int turn = 0;
    const uint32_t padded = (cols + 15) / 16 * 16, t0 = threadIdx.x * 8;
    constexpr int VPT = EPT ? EPT / 8 : 1;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const void *const from = row_of(x, row, ldx, F32 ? 4 : 2);
        Raw<F32> held[VPT];
        float m[1] = {0.0f};
        auto take = [&](Raw<F32> &r, uint32_t c) {
            r = Raw<F32>{};
            if (c < cols) fetch8<F32, WIDE>(r, from, c, cols);
        };
        auto look = [&](Raw<F32> &r, uint32_t c) {
            settle8<F32, WIDE>(r, c, cols);
#pragma unroll
            for (int e = 0; e < 8; ++e) m[0] = MaxBits::join(m[0], fabsf(raw_at(r, e)));
        };
        if constexpr (EPT) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) take(held[k], t0 + k * THREADS * 8);
#pragma unroll
            for (int k = 0; k < VPT; ++k) look(held[k], t0 + k * THREADS * 8);
        } else {
            for (uint32_t c = t0; c < cols; c += THREADS * 8) {
                take(held[0], c);
                look(held[0], c);
            }
        }
        block_join<MaxBits, THREADS, 1>(m, slots, turn);
        const QuantRow k = quant_row(m[0]);
        if (threadIdx.x == 0) scale[row] = k.scale;
        int8_t *const to = q + row * ldq;
        // (the padding is whole runs of 8)
        auto put = [&](const Raw<F32> &r, uint32_t c) {
            if (c < padded) quant8<WIDE>(k, to, c, padded, [&](int e) { return raw_at(r, e); });
        };
        if constexpr (EPT) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) put(held[i], t0 + i * THREADS * 8);
        } else {
            for (uint32_t c = t0; c < padded; c += THREADS * 8) {
                take(held[0], c);
                settle8<F32, WIDE>(held[0], c, cols);
                put(held[0], c);
            }
        }
    }
}

template <int BM, int BN, int WGM, int WGN, int SA, int SB>
hipError_t launch_tile(const Q8Args &q, hipStream_t s) {
    using T = Tile<i32x16_t, BM, BN, WGM, WGN, false, false, SA, SB>;
    return launch_lds<q8_tile_kernel<BM, BN, WGM, WGN, SA, SB>>(
        ((q.M + BM - 1) / BM) * ((q.N + BN - 1) / BN), T::THREADS, T::LDS_BYTES, s, q);
}

template <int MB, int NB, int NW, int S>
hipError_t launch_rows(const Q8Args &q, hipStream_t s) {
    using R = RowsKernel<MB, NB, NW, S>;
    return launch_lds<q8_rows_kernel<MB, NB, NW, S>>((q.N + NB * 16 - 1) / (NB * 16), NW * 64, R::LDS_BYTES, s, q);
}

hipError_t launch_rows_of(const Q8Args &q, hipStream_t s) {
    switch (q8_choice(q.M, q.N)) {
    case kQ8Rows16: return launch_rows<1, 1, 8, 4>(q, s);
    case kQ8Rows16Wide: return launch_rows<1, 2, 8, 3>(q, s);
    case kQ8Rows32: return launch_rows<2, 1, 8, 3>(q, s);
    case kQ8Rows32Wide: return launch_rows<2, 2, 8, 2>(q, s);
    case kQ8Rows64: return launch_rows<4, 1, 8, 2>(q, s);
    case kQ8Rows64Wide: return launch_rows<4, 2, 4, 3>(q, s);
    case kQ8Tile256: return launch_tile<256, 256, 2, 4, 2, 2>(q, s);
    case kQ8Tile128: return launch_tile<128, 128, 2, 4, 2, 3>(q, s);
    case kQ8Tile128Deep: return launch_tile<128, 128, 2, 4, 4, 4>(q, s);
    case kQ8Tile64x128: return launch_tile<64, 128, 2, 2, 2, 2>(q, s);
    case kQ8Tile64x128Deep: return launch_tile<64, 128, 2, 2, 3, 3>(q, s);
    default: return launch_tile<64, 64, 2, 2, 4, 4>(q, s);
    }
}

// All rows, in as many launches as they take.
hipError_t launch_product(const Q8Args &all, hipStream_t s) {
    const int64_t most = rows_of_launch(all.N);
    for (int64_t r = 0; r < all.M; r += most) {
        Q8Args q = all;
        q.M = all.M - r < most ? all.M - r : most;
        q.a += r * q.lda;
        q.a_scale += r;
        q.D = (char *)q.D + r * q.ldd * (q.out_f32 ? 4 : 2);
        const hipError_t e = launch_rows_of(q, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
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
    if (own(hipGetDevice(&p->device)) != hipSuccess) {
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
    // (arrays of no rows need not have an address)
    if ((rows > 0 && (!a || !a_scale || !D)) || !w || !w_scale || (bias != nullptr) != (d.has_bias != 0))
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
    q.wide_out = d.N % 8 == 0 && d.ldd % 8 == 0 && aligned(D, 16);
    return launch_product(q, (hipStream_t)stream) == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int gemm_q8_quantize(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, void *q,
                     int64_t ldq, void *scale, void *stream) {
    if (!known_type(dtype) || rows < 0 || cols < 1 || ldx < cols || ldq < (cols + 15) / 16 * 16)
        return GEMM_RS_ERR_INVALID_ARG;
    if ((rows > 0 && (!x || !q || !scale)) || !aligned(x, type_bytes(dtype)) || !aligned(scale, 4))
        return GEMM_RS_ERR_INVALID_ARG;
    if (cols >= kMaxK || rows > INT32_MAX || ldx > INT32_MAX || ldq > INT32_MAX)
        return GEMM_RS_ERR_UNSUPPORTED;
    if (rows == 0) return GEMM_RS_OK;
    const bool vec = cols % 8 == 0 && ldx % 8 == 0 && ldq % 8 == 0 && aligned(x, 16) && aligned(q, 8);
    const dim3 grid((unsigned)(rows < 65536 ? rows : 65536));
    hipError_t e = hipSuccess;
    auto go = [&](auto *kernel, int threads) {
        e = launch(kernel, grid, threads, 0, (hipStream_t)stream, x, rows, (uint32_t)cols, ldx, (int8_t *)q, ldq,
                   (float *)scale);
    };
    auto of_type = [&](auto f32, auto wide) {
        constexpr bool F = decltype(f32)::value, W = decltype(wide)::value;
        switch (quant_choice(rows, cols)) {
        case kQuantWave: return go(quantize_kernel<F, W, 32, 64>, 64);
        case kQuant2048: return go(quantize_kernel<F, W, 8, 256>, 256);
        case kQuant8192: return go(quantize_kernel<F, W, 16, 512>, 512);
        case kQuant16384: return go(quantize_kernel<F, W, 16, 1024>, 1024);
        default: return go(quantize_kernel<F, W, 0, 256>, 256);
        }
    };
    if (dtype == GEMM_RS_F32) vec ? of_type(std::true_type{}, std::true_type{}) : of_type(std::true_type{}, std::false_type{});
    else vec ? of_type(std::false_type{}, std::true_type{}) : of_type(std::false_type{}, std::false_type{});
    return e == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
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
