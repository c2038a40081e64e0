// bfloat16 products grouped by expert (gemm_grouped.h).
//
// The group sizes are on the device only, so a launch has the most
// workgroups that any split of the rows over the experts can need (one
// partly filled row tile per expert) and each workgroup finds its tile from
// the offsets.
#include <stdlib.h>

#include "gemm_grouped.h"
#include "mma_tile.h"

using namespace gemm_rs::ffn;

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 23;
constexpr int kMaxE = 1024;

struct GroupedArgs {
    int64_t rows, N, K, lda, ldb, ldc;
    int32_t E, out_f32, accumulate;
    int32_t tiles_m, tiles_n;     // TN: tiles of K and N of one expert
    const uint16_t *A, *B;
    const int32_t *offsets;
    void *C;
    int32_t *err;
};

// Rows [lo, hi) of expert e, clipped to 0 <= lo <= hi <= rows.
__device__ __forceinline__ void group_rows(const GroupedArgs &p, int e, int32_t *lo, int32_t *hi) {
    const int32_t rows = (int32_t)p.rows;
    int32_t l = p.offsets[e], h = p.offsets[e + 1];
    l = l < 0 ? 0 : l;
    l = l > rows ? rows : l;
    h = h > rows ? rows : h;
    h = h < l ? l : h;
    *lo = l;
    *hi = h;
}

// Run by one wave of a launch: records the first expert whose offsets had to
// be clipped.
__device__ __forceinline__ void check_offsets(const GroupedArgs &p) {
    for (int e = threadIdx.x; e < p.E; e += 64) {
        const int32_t a = p.offsets[e], b = p.offsets[e + 1];
        if (a < 0 || b < a || b > p.rows)
            if (atomicCAS(&p.err[0], 0, GEMM_RS_ERR_PROTOCOL) == 0) {
                p.err[1] = e;
                p.err[2] = a;
                p.err[3] = b;
            }
    }
}

struct RowTile {
    int e;
    int32_t lo, hi;     // the expert's rows
    int32_t row0;       // the tile's first row
    int tn;             // column tile
};

// The tile of workgroup b for row tiles of bm rows, found by each wave for
// itself (64 experts at a time, a prefix sum over the lanes); false if there
// are fewer tiles.  Tiles run expert by expert; inside an expert, row tiles
// in groups of 8, a group column by column, so that the tiles that run
// together read few rows of A and columns of B.
__device__ __forceinline__ bool find_row_tile(const GroupedArgs &p, int bm, uint32_t b, RowTile *t) {
    const int lane = threadIdx.x & 63;
    const uint32_t tn = (uint32_t)p.tiles_n;
    auto turn = [&](int e0, uint32_t *rt, uint32_t *upto) {
        int32_t lo = 0, hi = 0;
        if (e0 + lane < p.E) group_rows(p, e0 + lane, &lo, &hi);
        *rt = ((uint32_t)(hi - lo) + (uint32_t)bm - 1u) / (uint32_t)bm;
        uint32_t v = *rt * tn;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t u = __shfl_up(v, d);
            if (lane >= d) v += u;
        }
        *upto = v;
    };
    uint32_t rt, upto, total = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        turn(e0, &rt, &upto);
        total += __shfl(upto, 63);
    }
    if (b >= total) return false;
    b = xcd_run(b, total);
    uint32_t before = 0;      // tiles of the experts of earlier turns
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        if (p.E > 64) turn(e0, &rt, &upto);
        const uint32_t end = upto + before;
        const uint64_t past = __ballot(end > b);
        if (past) {
            const int src = __builtin_ctzll(past);
            const uint32_t n = __shfl(rt, src);
            const uint32_t j = b - (__shfl(end, src) - n * tn);
            // overlapping (clipped) groups can wrap the 32-bit prefix: such
            // a tile is left out, every other lies inside its expert
            if (j >= n * tn) return false;
            t->e = __builtin_amdgcn_readfirstlane(e0 + src);
            group_rows(p, t->e, &t->lo, &t->hi);
            t->lo = __builtin_amdgcn_readfirstlane(t->lo);
            t->hi = __builtin_amdgcn_readfirstlane(t->hi);
            const uint32_t g = j / (8 * tn), in = j - g * 8 * tn;
            const uint32_t rows = n - g * 8 < 8 ? n - g * 8 : 8;
            t->tn = __builtin_amdgcn_readfirstlane(in / rows);
            t->row0 = t->lo + __builtin_amdgcn_readfirstlane((g * 8 + in % rows) * (uint32_t)bm);
            return true;
        }
        before += __shfl(upto, 63);
    }
    return false;
}

// Any size, stride and alignment: 64 x 64 outputs per workgroup, 32 x 32 per
// wave, 64 of the contraction at a time, elements one by one (coalesced along
// the operand's contiguous axis, zeros outside it) into LDS rows of 144 bytes.
template <int OP>
__global__ __launch_bounds__(256) void grouped_narrow_kernel(GroupedArgs p) {
    constexpr int PITCH = 72;      // elements
    __shared__ __attribute__((aligned(16))) uint16_t As[64 * PITCH], Bs[64 * PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (blockIdx.x == 0 && wave == 0) check_offsets(p);
    int32_t lo, hi;
    int64_t m0, n0, m_end, k_len;
    int e;
    if constexpr (OP == GEMM_GROUPED_TN) {
        const int tiles = p.tiles_m * p.tiles_n;
        e = blockIdx.x / tiles;
        const int t = blockIdx.x - e * tiles;
        group_rows(p, e, &lo, &hi);
        m0 = (int64_t)(t / p.tiles_n) * 64;
        n0 = (int64_t)(t % p.tiles_n) * 64;
        m_end = p.K;
        k_len = hi - lo;
    } else {
        RowTile t;
        if (!find_row_tile(p, 64, blockIdx.x, &t)) return;
        e = t.e;
        lo = t.lo;
        m0 = t.row0;
        m_end = t.hi;
        n0 = (int64_t)t.tn * 64;
        k_len = p.K;
    }
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    f32x16_t acc = {};
    for (int64_t k0 = 0; k0 < k_len; k0 += 64) {
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int fast = tid & 63, slow = i * 4 + (tid >> 6);
            uint16_t av = 0, bv = 0;
            // A
            const int am = OP == GEMM_GROUPED_TN ? fast : slow, ak = OP == GEMM_GROUPED_TN ? slow : fast;
            if (m0 + am < m_end && k0 + ak < k_len)
                av = OP == GEMM_GROUPED_TN ? p.A[(lo + k0 + ak) * p.lda + m0 + am]
                                           : p.A[(m0 + am) * p.lda + k0 + ak];
            As[am * PITCH + ak] = av;
            const int bn = OP == GEMM_GROUPED_NT ? slow : fast, bk = OP == GEMM_GROUPED_NT ? fast : slow;
            if (n0 + bn < p.N && k0 + bk < k_len)
                bv = OP == GEMM_GROUPED_NN   ? p.B[((int64_t)e * p.K + k0 + bk) * p.ldb + n0 + bn]
                     : OP == GEMM_GROUPED_NT ? p.B[((int64_t)e * p.N + n0 + bn) * p.ldb + k0 + bk]
                                             : p.B[(lo + k0 + bk) * p.ldb + n0 + bn];
            Bs[bn * PITCH + bk] = bv;
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int c = s * 16 + (lane >> 5) * 8;
            acc = mma(*(const i32x4_t *)(As + (wm + (lane & 31)) * PITCH + c),
                      *(const i32x4_t *)(Bs + (wn + (lane & 31)) * PITCH + c), acc);
        }
        __syncthreads();
    }
    const int64_t m = m0 + wm + (lane & 31);
    const int64_t out0 = OP == GEMM_GROUPED_TN ? ((int64_t)e * p.K + m) * p.ldc : m * p.ldc;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int64_t n = n0 + wn + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
        if (m < m_end && n < p.N) {
            float x = acc[v];
            if (p.out_f32) {
                float *c = (float *)p.C + out0 + n;
                *c = p.accumulate ? *c + x : x;
            } else {
                uint16_t *c = (uint16_t *)p.C + out0 + n;
                if (p.accumulate) x += bf16_lo(*c);
                *c = (uint16_t)to_bf16(x);
            }
        }
    }
}

// 8 columns of a row of C.
__device__ __forceinline__ void store8(const GroupedArgs &p, int64_t row, int64_t n, const int (&v)[8]) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __int_as_float(v[e]);
    const uint32_t at = (uint32_t)n;
    void *const C = row_of(p.C, row, p.ldc, p.out_f32 ? 4 : 2);
    if (p.out_f32) {
        if (p.accumulate) {
            Raw<true, 8> c;
            load_raw(c, C, at);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += raw_at(c, e);
        }
        store_vec<true, 8>(C, at, x);
    } else {
        if (p.accumulate) {
            Raw<false, 8> c;
            load_raw(c, C, at);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += raw_at(c, e);
        }
        store_vec<false, 8>(C, at, x);
    }
}

// Sizes, strides and addresses that are multiples of 8 elements.
template <int OP, int BM, int BN, int WGM, int WGN, int STAGES>
using GroupedTile = Tile<f32x16_t, BM, BN, WGM, WGN, OP == GEMM_GROUPED_TN, OP != GEMM_GROUPED_NT, STAGES>;

template <int OP, int BM, int BN, int WGM, int WGN, int STAGES>
__global__ __launch_bounds__(64 * WGM * WGN) void grouped_tile_kernel(GroupedArgs p) {
    using T = GroupedTile<OP, BM, BN, WGM, WGN, STAGES>;
    extern __shared__ __attribute__((aligned(1024))) char smem_generic[];
    lds_t *smem = (lds_t *)smem_generic;
    if (blockIdx.x == 0 && threadIdx.x < 64) check_offsets(p);
    T tile;
    if constexpr (OP == GEMM_GROUPED_TN) {
        // XCD x takes the x-th eighth of every expert's tiles, so the XCDs'
        // shares are equal however uneven the groups are
        const int tiles = p.tiles_m * p.tiles_n, per = (tiles + 7) / 8;
        const int j = blockIdx.x / 8, e = j / per;
        const int t = (int)(blockIdx.x % 8) * per + (j - e * per);
        if (t >= tiles) return;
        const int64_t m0 = (int64_t)(t / p.tiles_n) * BM, n0 = (int64_t)(t % p.tiles_n) * BN;
        int32_t lo, hi;
        group_rows(p, e, &lo, &hi);
        lo = __builtin_amdgcn_readfirstlane(lo);
        hi = __builtin_amdgcn_readfirstlane(hi);
        if (hi == lo && p.accumulate) return;
        const int32_t m_left = (int32_t)(p.K - m0 < BM ? p.K - m0 : BM);
        const int32_t n_left = (int32_t)(p.N - n0 < BN ? p.N - n0 : BN);
        const Operand a = {(const char *)(p.A + (int64_t)lo * p.lda + m0), p.lda * 2, m_left * 2};
        const Operand b = {(const char *)(p.B + (int64_t)lo * p.ldb + n0), p.ldb * 2, n_left * 2};
        tile.template run<2>(smem, a, b, hi - lo);
        tile.template store<8>(smem, [&](int r, int c, const int (&v)[8]) {
            if (r < m_left && c < n_left) store8(p, (int64_t)e * p.K + m0 + r, n0 + c, v);
        });
    } else {
        RowTile t;
        if (!find_row_tile(p, BM, blockIdx.x, &t)) return;
        const int64_t n0 = (int64_t)t.tn * BN;
        const int32_t m_left = t.hi - t.row0 < BM ? t.hi - t.row0 : BM;
        const int32_t n_left = (int32_t)(p.N - n0 < BN ? p.N - n0 : BN);
        const Operand a = {(const char *)(p.A + (int64_t)t.row0 * p.lda), p.lda * 2, m_left};
        const Operand b = OP == GEMM_GROUPED_NN
            ? Operand{(const char *)(p.B + (int64_t)t.e * p.K * p.ldb + n0), p.ldb * 2, n_left * 2}
            : Operand{(const char *)(p.B + ((int64_t)t.e * p.N + n0) * p.ldb), p.ldb * 2, n_left};
        tile.template run<2>(smem, a, b, (int32_t)p.K);
        tile.template store<8>(smem, [&](int r, int c, const int (&v)[8]) {
            if (r < m_left && c < n_left) store8(p, (int64_t)t.row0 + r, n0 + c, v);
        });
    }
}

template <int OP, int BM, int BN, int WGM, int WGN, int STAGES>
hipError_t launch_tile(GroupedArgs &a, hipStream_t s) {
    using T = GroupedTile<OP, BM, BN, WGM, WGN, STAGES>;
    a.tiles_n = (int32_t)((a.N + BN - 1) / BN);
    a.tiles_m = (int32_t)((a.K + BM - 1) / BM);
    int64_t blocks;
    if (OP == GEMM_GROUPED_TN) blocks = (((int64_t)a.tiles_m * a.tiles_n + 7) / 8) * 8 * a.E;
    else blocks = (a.rows / BM + (a.E < a.rows ? a.E : a.rows)) * a.tiles_n;
    return launch_lds<grouped_tile_kernel<OP, BM, BN, WGM, WGN, STAGES>>(blocks, T::THREADS, T::LDS_BYTES, s, a);
}

template <int OP>
hipError_t launch_op(GroupedArgs &a, bool wide, hipStream_t s) {
    if (!wide) {
        a.tiles_n = (int32_t)((a.N + 63) / 64);
        a.tiles_m = (int32_t)((a.K + 63) / 64);
        const int64_t row_tiles = OP == GEMM_GROUPED_TN ? (int64_t)a.E * a.tiles_m
                                                        : a.rows / 64 + (a.E < a.rows ? a.E : a.rows);
        hipLaunchKernelGGL(grouped_narrow_kernel<OP>, dim3((unsigned)(row_tiles * a.tiles_n)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    if constexpr (OP == GEMM_GROUPED_TN) {
        const int64_t big = (int64_t)a.E * ((a.K + 255) / 256) * ((a.N + 255) / 256);
        if (big >= kCus) return launch_tile<OP, 256, 256, 2, 4, 2>(a, s);
        return launch_tile<OP, 128, 128, 2, 2, 4>(a, s);
    } else {
        const int64_t avg = a.rows / a.E;      // the sizes themselves are on the device
        if (avg >= 192) return launch_tile<OP, 256, 256, 2, 4, 2>(a, s);
        if (avg >= 48) return launch_tile<OP, 128, 128, 2, 2, 4>(a, s);
        return launch_tile<OP, 32, 128, 1, 4, 6>(a, s);
    }
}

int validate(const gemm_grouped_desc_t &d) {
    if (d.M < 1 || d.N < 1 || d.K < 1 || d.E < 1 || d.pad != 0) return GEMM_RS_ERR_INVALID_ARG;
    if (d.op < GEMM_GROUPED_NN || d.op > GEMM_GROUPED_TN || !known_type(d.out_dtype))
        return GEMM_RS_ERR_INVALID_ARG;
    if ((d.accumulate != 0 && d.accumulate != 1) || (d.accumulate && d.op != GEMM_GROUPED_TN))
        return GEMM_RS_ERR_INVALID_ARG;
    const int64_t bcols = d.op == GEMM_GROUPED_NT ? d.K : d.N;
    if (d.lda < 0 || d.ldb < 0 || d.ldc < 0 || (d.lda && d.lda < d.K) || (d.ldb && d.ldb < bcols) ||
        (d.ldc && d.ldc < d.N))
        return GEMM_RS_ERR_INVALID_ARG;
    if (d.E > kMaxE || d.M > INT32_MAX || d.N > INT32_MAX || d.K > INT32_MAX)
        return GEMM_RS_ERR_UNSUPPORTED;
    if (d.lda >= kMaxStride || d.ldb >= kMaxStride || d.ldc >= kMaxStride || d.K >= kMaxStride ||
        d.N >= kMaxStride)
        return GEMM_RS_ERR_UNSUPPORTED;
    // most tiles of the narrow kernel, which has the smallest
    const int64_t tm = d.op == GEMM_GROUPED_TN ? d.E * ((d.K + 63) / 64) : d.M / 64 + d.E;
    if (tm * ((d.N + 63) / 64) > INT32_MAX) return GEMM_RS_ERR_UNSUPPORTED;
    return GEMM_RS_OK;
}

}  // namespace

struct gemm_grouped_plan_s {
    gemm_grouped_desc_t d;    // strides filled in
    int device;
    int32_t *err;
};

extern "C" {

int gemm_grouped_plan(const gemm_grouped_desc_t *desc, gemm_grouped_plan_t *out) {
    if (!desc || !out) return GEMM_RS_ERR_INVALID_ARG;
    *out = nullptr;
    const int rc = validate(*desc);
    if (rc != GEMM_RS_OK) return rc;
    gemm_grouped_plan_s *p = (gemm_grouped_plan_s *)calloc(1, sizeof(gemm_grouped_plan_s));
    if (!p) return GEMM_RS_ERR_HIP;
    p->d = *desc;
    if (!p->d.lda) p->d.lda = p->d.K;
    if (!p->d.ldb) p->d.ldb = p->d.op == GEMM_GROUPED_NT ? p->d.K : p->d.N;
    if (!p->d.ldc) p->d.ldc = p->d.N;
    hipError_t e = hipGetDevice(&p->device);
    if (e == hipSuccess) e = hipMalloc((void **)&p->err, 16);
    // a blocking copy: the word is zero before any later launch on any stream
    const int32_t zero[4] = {0, 0, 0, 0};
    if (e == hipSuccess) e = hipMemcpy(p->err, zero, 16, hipMemcpyHostToDevice);
    if (e != hipSuccess) {
        if (p->err) (void)hipFree(p->err);
        free(p);
        return GEMM_RS_ERR_HIP;
    }
    *out = p;
    return GEMM_RS_OK;
}

int gemm_grouped_run(gemm_grouped_plan_t p, const void *A, const void *B, const void *offsets,
                     void *C, int64_t rows, void *stream) {
    if (!p || !on_device(p->device)) return GEMM_RS_ERR_INVALID_ARG;
    const gemm_grouped_desc_t &d = p->d;
    if (rows < 0 || rows > d.M) return GEMM_RS_ERR_INVALID_ARG;
    if (!A || !B || !offsets || !C || !aligned(A, 2) || !aligned(B, 2) || !aligned(offsets, 4) ||
        !aligned(C, type_bytes(d.out_dtype)))
        return GEMM_RS_ERR_INVALID_ARG;
    if (rows == 0 && d.op != GEMM_GROUPED_TN) return GEMM_RS_OK;
    GroupedArgs a = {};
    a.rows = rows;
    a.N = d.N;
    a.K = d.K;
    a.lda = d.lda;
    a.ldb = d.ldb;
    a.ldc = d.ldc;
    a.E = d.E;
    a.out_f32 = d.out_dtype == GEMM_RS_F32;
    a.accumulate = d.accumulate;
    a.A = (const uint16_t *)A;
    a.B = (const uint16_t *)B;
    a.offsets = (const int32_t *)offsets;
    a.C = C;
    a.err = p->err;
    hipStream_t s = (hipStream_t)stream;
    const int64_t c_elems = d.out_dtype == GEMM_RS_F32 ? 4 : 8;
    const bool wide = d.N % 8 == 0 && d.K % 8 == 0 && d.lda % 8 == 0 && d.ldb % 8 == 0 &&
                      d.ldc % c_elems == 0 && aligned(A, 16) && aligned(B, 16) && aligned(C, 16);
    const hipError_t e = d.op == GEMM_GROUPED_NN   ? launch_op<GEMM_GROUPED_NN>(a, wide, s)
                         : d.op == GEMM_GROUPED_NT ? launch_op<GEMM_GROUPED_NT>(a, wide, s)
                                                   : launch_op<GEMM_GROUPED_TN>(a, wide, s);
    return e == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int gemm_grouped_status(gemm_grouped_plan_t p, void *stream, int32_t *detail) {
    if (!p || !on_device(p->device)) return GEMM_RS_ERR_INVALID_ARG;
    int32_t h[4] = {0, 0, 0, 0};
    hipError_t e = hipStreamSynchronize((hipStream_t)stream);
    if (e == hipSuccess) e = hipMemcpy(h, p->err, 16, hipMemcpyDeviceToHost);
    const int32_t zero[4] = {0, 0, 0, 0};
    if (e == hipSuccess && h[0] != 0) e = hipMemcpy(p->err, zero, 16, hipMemcpyHostToDevice);
    if (e != hipSuccess) return GEMM_RS_ERR_HIP;
    if (detail)
        for (int i = 0; i < 4; ++i) detail[i] = h[i];
    return h[0];
}

int gemm_grouped_query(gemm_grouped_plan_t p, gemm_grouped_info_t *info) {
    if (!p || !info) return GEMM_RS_ERR_INVALID_ARG;
    info->workspace_bytes = 16;
    return GEMM_RS_OK;
}

int gemm_grouped_destroy(gemm_grouped_plan_t p) {
    if (!p) return GEMM_RS_OK;
    int cur = -1;
    bool switched = false;
    if (hipGetDevice(&cur) == hipSuccess && cur != p->device)
        switched = hipSetDevice(p->device) == hipSuccess;
    // teardown is best effort: a failure here leaves nothing to undo
    (void)hipFree(p->err);
    if (switched) (void)hipSetDevice(cur);
    free(p);
    return GEMM_RS_OK;
}

}  // extern "C"
