// bfloat16 products grouped by expert (gemm_grouped.h).
//
// The group sizes are on the device only, so a launch has the most
// workgroups that any split of the rows over the experts can need (one
// partly filled row tile per expert) and each workgroup finds its tile from
// the offsets.
//
// Bound by the matrix pipe at the board's power limit where experts have many
// rows (16384 rows, 8 experts of 4096 x 3584: product 437 us, 1100 TFLOP/s,
// gradients 466 and 420 us), by reading B or writing weight gradients where they
// have few (8000 rows in uneven groups, 64 experts of 4096 x 1792, inputs in turn:
// 218 us, 4.7 TB/s; 128 rows, 8 experts of 4096 x 3584: 44 us, 5.4 TB/s, part of it
// from the caches; gradients of 44 experts of 4040 x 2048 in 32 bits, 164 rows: 223
// us, 6.5 TB/s).
#include <stdlib.h>

#include "gemm_grouped.h"
#include "mma_tile.h"

using namespace gemm_rs::ffn;

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 23;
constexpr int kMaxE = 1024;
// most rows: the last step of 64 that is begun (some are loaded ahead) ends
// within 32 bits
constexpr int64_t kMaxRows = INT32_MAX - 1024;

struct GroupedArgs {
    int64_t rows, N, K, lda, ldb, ldc;
    int32_t E, out_f32, accumulate;
    int32_t tiles_m, tiles_n;     // TN: tiles of K and N of one expert
    const uint16_t *A, *B;
    const int32_t *offsets;
    void *C;
    int32_t *err;
    int32_t parts;                // TN: workgroups that share a tile's contraction
    float *slots;                 // their sums, [part][E][K][N] (parts > 1)
    int32_t stream;               // TN: C is stored past the caches
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

// Run by one wave of a launch: records an expert whose offsets had to be clipped
// (of several, whichever lane's exchange comes first), unless one is recorded.
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
    int32_t row0;       // the tile's first row
    int32_t end;        // past the expert's last row
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
            int32_t lo, hi;
            group_rows(p, t->e, &lo, &hi);
            t->end = __builtin_amdgcn_readfirstlane(hi);
            const uint32_t g = j / (8 * tn), in = j - g * 8 * tn;
            const uint32_t rows = n - g * 8 < 8 ? n - g * 8 : 8;
            t->tn = __builtin_amdgcn_readfirstlane(in / rows);
            t->row0 = __builtin_amdgcn_readfirstlane(lo + (int32_t)((g * 8 + in % rows) * (uint32_t)bm));
            return true;
        }
        before += __shfl(upto, 63);
    }
    return false;
}

// 4 or 8 columns of a row of C; STREAM: past the caches.
template <bool WIDE, bool STREAM>
__device__ __forceinline__ void store_four(const GroupedArgs &p, int64_t row, int64_t n, const int *v) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __int_as_float(v[e]);
    float *const C = (float *)row_of(p.C, row, p.ldc, 4);
    const uint32_t at = (uint32_t)n, cols = (uint32_t)p.N;
    if (p.accumulate) {
        typedef std::conditional_t<WIDE, u32x4_t, u32x4_at4_t> words;
        if (WIDE || at + 4 <= cols) {
            const u32x4_t c = *(const words *)(C + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += __uint_as_float(c[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (at + e < cols) x[e] += C[at + e];
        }
    }
    store4<WIDE, STREAM>(C, at, cols, x);
}
template <bool WIDE, bool STREAM>
__device__ __forceinline__ void store_run(const GroupedArgs &p, int64_t row, int64_t n, const int (&v)[8]) {
    if (p.out_f32) {
        store_four<WIDE, STREAM>(p, row, n, v);
        if (WIDE || n + 4 < p.N) store_four<WIDE, STREAM>(p, row, n + 4, v + 4);
        return;
    }
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __int_as_float(v[e]);
    const uint32_t at = (uint32_t)n, cols = (uint32_t)p.N;
    void *const C = row_of(p.C, row, p.ldc, 2);
    if (p.accumulate) {
        Raw<false> c;
        load8<false, WIDE>(c, C, at, cols);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += raw_at(c, e);
    }
    store8<false, WIDE, STREAM>(C, at, cols, x);
}

// Operands of 64 of the contraction in 128-byte LDS rows, for the kernels of
// small tiles: 16-byte chunk c of row r sits at c ^ swz.  Row operand (a row of
// the tile per output row): a lane's fragment of slice ks is 16 bytes of row
// m + lane % 32.  Column operand (a row of the tile per row of the contraction):
// two transposing reads, each of 4 rows of 4 chunks.
__device__ __forceinline__ int row_swz(int r) { return (r ^ (r >> 3)) & 7; }
__device__ __forceinline__ int col_swz(int r) { return 4 * ((r >> 1) & 1); }
template <bool COL>
__device__ __forceinline__ int swz(int r) { return COL ? col_swz(r) : row_swz(r); }
template <bool COL>
__device__ __forceinline__ i32x4_t fragment(lds_t *tile, int m, int ks) {
    typedef __attribute__((address_space(3))) i32x4_t lds_i32x4;
    typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
    const int lane = threadIdx.x & 63;
    if constexpr (COL) {
        const int grp = lane >> 4, te = (lane & 15) >> 2, tq = lane & 3;
        const int r = ks * 16 + 8 * (grp >> 1) + te, x = m + 16 * (grp & 1) + 4 * tq;
        // rows r and r + 4 have the same swizzle
        lds_t *const q = tile + r * 128 + (((x >> 3) ^ col_swz(r)) << 4) + ((x & 7) << 1);
        const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)q);
        const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(q + 4 * 128));
        return __builtin_bit_cast(i32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        const int r = m + (lane & 31);
        return *(lds_i32x4 *)(tile + r * 128 + (((2 * ks + (lane >> 5)) ^ row_swz(r)) << 4));
    }
}

// Any size, stride and alignment, for what the others do not take: 64 x 64
// outputs per workgroup, 32 x 32 per wave, 64 of the contraction at a time,
// loaded through registers (16 bytes at any element address, zeros outside the
// operand) two steps ahead, and written to the other of two LDS buffers one step
// ahead.  Even groups, repeated calls: 8000 rows, 64 experts of 4095 x 1791: product
// and gradient of x 450 us, 260 TFLOP/s (loads of single elements took 2350), of
// 4096 x 1792 in the tiles below 190 and 200; 16384 rows, 8 experts of 4095 x 3583 1.4 ms, 340 TFLOP/s, of
// 4096 x 3584 0.4.  Bound by the latency of a step, as a tile of this size has few
// loads to run ahead.
template <int OP>
__global__ __launch_bounds__(256) void grouped_narrow_kernel(GroupedArgs p) {
    constexpr bool A_COL = OP == GEMM_GROUPED_TN, B_COL = OP != GEMM_GROUPED_NT;
    __shared__ __attribute__((aligned(1024))) char smem_generic[4 * 8192];
    lds_t *const smem = (lds_t *)smem_generic;      // [buffer][operand]
    typedef __attribute__((address_space(3))) u32x4_t lds_u32x4;
    typedef __attribute__((address_space(3))) f32x4_t lds_f32x4;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (blockIdx.x == 0 && wave == 0) check_offsets(p);
    int32_t lo = 0, hi;
    int64_t m0, n0, m_end, k_len;
    int e;
    if constexpr (OP == GEMM_GROUPED_TN) {
        const int tiles = p.tiles_m * p.tiles_n;
        e = blockIdx.x / tiles;
        const int t = blockIdx.x - e * tiles;
        group_rows(p, e, &lo, &hi);
        m0 = (int64_t)(t / p.tiles_n) * 64;
        n0 = (int64_t)(t % p.tiles_n) * 64;
        if (hi == lo && p.accumulate) return;
        m_end = p.K;
        k_len = hi - lo;
    } else {
        RowTile t;
        if (!find_row_tile(p, 64, blockIdx.x, &t)) return;
        e = t.e;
        m0 = t.row0;
        m_end = t.end;
        n0 = (int64_t)t.tn * 64;
        k_len = p.K;
    }
    // this thread's chunks: number tid % 8 of rows tid / 8 and 32 further
    const int chunk = tid & 7;
    Raw<false> ra[2][2], rb[2][2];                  // of two steps
    auto take = [&](Raw<false> &r, const uint16_t *at, int64_t ld, int64_t row, int64_t rows,
                    int64_t from, int64_t upto) __attribute__((always_inline)) {
        r = Raw<false>{};
        if (row < rows && from + chunk * 8 < upto)
            fetch8<false, false>(r, at + row * ld, (uint32_t)from + chunk * 8, (uint32_t)upto);
    };
    auto fetch = [&](int set, int64_t k0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (tid >> 3) + 32 * i;
            if constexpr (A_COL) take(ra[set][i], p.A + (int64_t)lo * p.lda, p.lda, k0 + r, k_len, m0, m_end);
            else take(ra[set][i], p.A, p.lda, m0 + r, m_end, k0, k_len);
            if constexpr (OP == GEMM_GROUPED_NN)
                take(rb[set][i], p.B + (int64_t)e * p.K * p.ldb, p.ldb, k0 + r, k_len, n0, p.N);
            else if constexpr (OP == GEMM_GROUPED_TN)
                take(rb[set][i], p.B + (int64_t)lo * p.ldb, p.ldb, k0 + r, k_len, n0, p.N);
            else take(rb[set][i], p.B + (int64_t)e * p.N * p.ldb, p.ldb, n0 + r, p.N, k0, k_len);
        }
    };
    // (rows past an operand's hold zeros, which the shift leaves)
    auto put = [&](int set, int64_t k0) __attribute__((always_inline)) {
        const uint32_t a_from = (uint32_t)(A_COL ? m0 : k0) + chunk * 8, b_from = (uint32_t)(B_COL ? n0 : k0) + chunk * 8;
        const uint32_t a_upto = (uint32_t)(A_COL ? m_end : k_len), b_upto = (uint32_t)(B_COL ? p.N : k_len);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (tid >> 3) + 32 * i;
            settle8<false, false>(ra[set][i], a_from, a_upto);
            settle8<false, false>(rb[set][i], b_from, b_upto);
            lds_t *const at = smem + set * 16384 + r * 128;
            *(lds_u32x4 *)(at + ((chunk ^ swz<A_COL>(r)) << 4)) = ra[set][i].a;
            *(lds_u32x4 *)(at + 8192 + ((chunk ^ swz<B_COL>(r)) << 4)) = rb[set][i].a;
        }
    };
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    f32x16_t acc = {};
    fetch(0, 0);
    fetch(1, 64);                                   // (nothing past the end)
    put(0, 0);
    lds_only_barrier();
    // the step at k0, in buffer `now`
    auto step = [&](int now, int64_t k0) __attribute__((always_inline)) {
        fetch(now, k0 + 128);
        lds_t *const at = smem + now * 16384;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            acc = mma(fragment<A_COL>(at, wm, ks), fragment<B_COL>(at + 8192, wn, ks), acc);
        put(now ^ 1, k0 + 64);
        lds_only_barrier();
    };
    for (int64_t k0 = 0; k0 < k_len; k0 += 128) {
        step(0, k0);
        if (k0 + 64 < k_len) step(1, k0 + 64);
    }
    // through LDS, so that runs of 8 columns are stored together
    const int m = wm + (lane & 31);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const f32x4_t v = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
        *(lds_f32x4 *)(smem + m * 256 + (((wn / 4 + 2 * q + (lane >> 5)) ^ (m & 15)) << 4)) = v;
    }
    lds_only_barrier();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = (tid >> 3) + 32 * i, c = chunk * 8;
        if (m0 + r >= m_end || n0 + c >= p.N) continue;
        int v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4_t x = *(lds_f32x4 *)(smem + r * 256 + (((2 * chunk + h) ^ (r & 15)) << 4));
#pragma unroll
            for (int u = 0; u < 4; ++u) v[4 * h + u] = __float_as_int(x[u]);
        }
        store_run<false, false>(p, (OP == GEMM_GROUPED_TN ? (int64_t)e * p.K : 0) + m0 + r, n0 + c, v);
    }
}

// Sizes, strides and addresses that are multiples of 8 elements.
template <int OP, int BM, int BN, int WGM, int WGN, int SA, int SB>
using GroupedTile = Tile<f32x16_t, BM, BN, WGM, WGN, OP == GEMM_GROUPED_TN, OP != GEMM_GROUPED_NT, SA, SB>;

// A from the tile's first row, and expert e's B from column n0 (NN, NT).
__device__ __forceinline__ Operand row_operand(const GroupedArgs &p, const RowTile &t, int32_t rows) {
    return {(const char *)(p.A + (int64_t)t.row0 * p.lda), p.lda * 2, rows};
}
template <int OP>
__device__ __forceinline__ Operand column_operand(const GroupedArgs &p, int e, int64_t n0, int32_t cols) {
    if constexpr (OP == GEMM_GROUPED_NN)
        return {(const char *)(p.B + (int64_t)e * p.K * p.ldb + n0), p.ldb * 2, cols * 2};
    else
        return {(const char *)(p.B + ((int64_t)e * p.N + n0) * p.ldb), p.ldb * 2, cols};
}

// A tile's m_left x n_left (columns: a multiple of 8) outputs from row m0 and column n0 of C.
template <bool STREAM, class T>
__device__ __forceinline__ void store_tile(const GroupedArgs &p, const T &tile, lds_t *smem, int64_t m0, int32_t m_left,
                                           int64_t n0, int32_t n_left) {
    if (p.out_f32)
        tile.template store<true>(smem, [&](int r, int c, int d, const int (&v)[8]) {
            if (r < m_left && c < n_left) store_four<true, STREAM>(p, m0 + r, n0 + c, v);
            if (r < m_left && d < n_left) store_four<true, STREAM>(p, m0 + r, n0 + d, v + 4);
        });
    else
        tile.template store<false>(smem, [&](int r, int c, int, const int (&v)[8]) {
            if (r < m_left && c < n_left) store_run<true, STREAM>(p, m0 + r, n0 + c, v);
        });
}

template <int OP, int BM, int BN, int WGM, int WGN, int SA, int SB>
__global__ __launch_bounds__(64 * WGM * WGN) void grouped_tile_kernel(GroupedArgs p) {
    using T = GroupedTile<OP, BM, BN, WGM, WGN, SA, SB>;
    extern __shared__ __attribute__((aligned(1024))) char smem_generic[];
    lds_t *smem = (lds_t *)smem_generic;
    if (blockIdx.x == 0 && threadIdx.x < 64) check_offsets(p);
    T tile;
    if constexpr (OP == GEMM_GROUPED_TN) {
        // Each XCD takes an eighth of every expert's tiles, so that the shares
        // are equal however uneven the groups are, another one for the next
        // expert, as eighths differ by a tile; part by part, so that few XCDs
        // read the same rows.
        const int of_part = p.tiles_m * p.tiles_n, tiles = of_part * p.parts, per = (tiles + 7) / 8;
        const int j = blockIdx.x / 8, e = j / per, eighth = (int)(blockIdx.x + e) % 8;
        const int u = (int)((int64_t)tiles * eighth / 8) + (j - e * per);
        if (u >= (int)((int64_t)tiles * (eighth + 1) / 8)) return;
        const int part = u / of_part, t = u - part * of_part;
        const int64_t m0 = (int64_t)(t / p.tiles_n) * BM, n0 = (int64_t)(t % p.tiles_n) * BN;
        int32_t lo, hi;
        group_rows(p, e, &lo, &hi);
        lo = __builtin_amdgcn_readfirstlane(lo);
        hi = __builtin_amdgcn_readfirstlane(hi);
        if (hi == lo && p.accumulate && p.parts == 1) return;
        const int32_t m_left = (int32_t)(p.K - m0 < BM ? p.K - m0 : BM);
        const int32_t n_left = (int32_t)(p.N - n0 < BN ? p.N - n0 : BN);
        GroupedArgs out = p;
        if (p.parts > 1) {
            const uint32_t steps = (uint32_t)T::template steps_of<2>(hi - lo);
            const int32_t end = lo + (int32_t)((uint64_t)(part + 1) * steps / p.parts) * 64;
            lo += (int32_t)((uint64_t)part * steps / p.parts) * 64;
            hi = hi < end ? hi : end;
            out.C = p.slots + (int64_t)part * p.E * p.K * p.N;
            out.ldc = p.N;
            out.out_f32 = 1;
            out.accumulate = 0;
        }
        const Operand a = {(const char *)(p.A + (int64_t)lo * p.lda + m0), p.lda * 2, m_left * 2};
        const Operand b = {(const char *)(p.B + (int64_t)lo * p.ldb + n0), p.ldb * 2, n_left * 2};
        tile.template run<2>(smem, a, b, hi - lo);
        if (p.stream) store_tile<true>(out, tile, smem, (int64_t)e * p.K + m0, m_left, n0, n_left);
        else store_tile<false>(out, tile, smem, (int64_t)e * p.K + m0, m_left, n0, n_left);
    } else {
        RowTile t;
        if (!find_row_tile(p, BM, blockIdx.x, &t)) return;
        const int64_t n0 = (int64_t)t.tn * BN;
        const int32_t m_left = t.end - t.row0 < BM ? t.end - t.row0 : BM;
        const int32_t n_left = (int32_t)(p.N - n0 < BN ? p.N - n0 : BN);
        tile.template run<2>(smem, row_operand(p, t, m_left), column_operand<OP>(p, t.e, n0, n_left), (int32_t)p.K);
        store_tile<false>(p, tile, smem, t.row0, m_left, n0, n_left);
    }
}

// Few rows per expert (NN, NT): 32 rows and 64 columns per workgroup.  Bound by
// streaming B, so the contraction is dealt out to the 4 waves 64 at a time and
// each wave streams its share through 3 stages of LDS of its own: no wave waits
// for another until their sums meet, in the order of the waves.  32 rows of one
// expert, K = 4096, N = 3584: 16 us, 1.8 TB/s of B (a 128 x 128 tile 25 us).
template <int OP>
struct StreamTile {
    static constexpr int BM = 32, BN = 64, FN = BN / 32, NW = 4, S = 3;
    static constexpr int A_LOADS = BM / 8, B_LOADS = BN / 8, LOADS = A_LOADS + B_LOADS;   // of 1 KB
    static constexpr int A_BYTES = A_LOADS * 1024, STAGE = LOADS * 1024;
    static constexpr int THREADS = NW * 64, LDS_BYTES = NW * S * STAGE;
    static constexpr bool COL = OP == GEMM_GROUPED_NN;
    static_assert(BN == 64, "B's rows of a stage are 128 bytes in both forms");
    static_assert(LDS_BYTES <= 160 * 1024 && BM * BN * 4 <= S * STAGE, "LDS");
    static_assert((S - 1) * LOADS < 64, "the load counter");

    template <class F>
    static __device__ __forceinline__ void run(lds_t *smem, const Operand &a, const Operand &b, int32_t K, F store) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int pieces = (int)(((uint32_t)K + 63) / 64);
        const int mine = pieces > wave ? (pieces - wave + NW - 1) / NW : 0;
        lds_t *const own = smem + wave * (S * STAGE);
        const uint32_t own_base = (uint32_t)(size_t)own;
        const int lr = lane >> 3, lc = lane & 7;
        // a lane's offset in load i: rows i * 8 + lr; the row swizzle takes 8
        // values over i, the column swizzle one
        auto issue = [&](int piece, int st) __attribute__((always_inline)) {
            const int k = (piece * NW + wave) * 64;
            const int left = K - k < 64 ? K - k : 64;
            const i32x4_t ra = buffer_of(a.base + (int64_t)k * 2, (uint32_t)(a.span - 1) * (uint32_t)a.ld + left * 2);
            const i32x4_t rb = COL ? buffer_of(b.base + (int64_t)k * b.ld, (uint32_t)(left - 1) * (uint32_t)b.ld + (uint32_t)b.span)
                                   : buffer_of(b.base + (int64_t)k * 2, (uint32_t)(b.span - 1) * (uint32_t)b.ld + left * 2);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const bool isb = i >= A_LOADS;
                const int r = (isb ? i - A_LOADS : i) * 8 + lr;
                const int c = lc ^ (isb ? swz<COL>(r) : row_swz(r));
                uint32_t v = (uint32_t)r * (uint32_t)(isb ? b.ld : a.ld) + c * 16;
                // past the contraction's end: rows of NN's B lie past the
                // descriptor, chunks of the others are sent there
                if (!(isb && COL) && c * 8 >= left) v = 0xfffffff0u;
                load_to_lds(isb ? rb : ra, v, own_base + st * STAGE + i * 1024);
            }
        };
        typedef __attribute__((address_space(3))) f32x4_t lds_f32x4;
        f32x16_t acc[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[j] = f32x16_t{};
#pragma unroll
        for (int s = 0; s < S - 1; ++s)
            if (s < mine) issue(s, s);
        int st = 0;
        for (int n = 0; n < mine; ++n) {
            wait_groups<LOADS, S - 2>(mine - 1 - n);
            if (n + S - 1 < mine) issue(n + S - 1, st == 0 ? S - 1 : st - 1);
            lds_t *const at = own + st * STAGE, *const bt = at + A_BYTES;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const i32x4_t af = fragment<false>(at, 0, ks);
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[j] = mma(af, fragment<COL>(bt, j * 32, ks), acc[j]);
            }
            // the reads are done before the next issue overwrites their stage
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (++st == S) st = 0;
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4_t v = {acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
                *(lds_f32x4 *)(own + ((lane & 31) * BN + j * 32 + 8 * q + 4 * (lane >> 5)) * 4) = v;
            }
        __syncthreads();
        for (int u = tid; u < BM * BN / 8; u += THREADS) {
            const int r = u / (BN / 8), c = u % (BN / 8) * 8;
            f32x4_t lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                lds_t *const q = smem + w * (S * STAGE) + (r * BN + c) * 4;
                lo += *(lds_f32x4 *)q;
                hi += *(lds_f32x4 *)(q + 16);
            }
            int v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = __float_as_int(lo[e]);
                v[e + 4] = __float_as_int(hi[e]);
            }
            store(r, c, v);
        }
    }
};

template <int OP>
__global__ __launch_bounds__(StreamTile<OP>::THREADS) void grouped_stream_kernel(GroupedArgs p) {
    using T = StreamTile<OP>;
    extern __shared__ __attribute__((aligned(1024))) char smem_generic[];
    if (blockIdx.x == 0 && threadIdx.x < 64) check_offsets(p);
    RowTile t;
    if (!find_row_tile(p, T::BM, blockIdx.x, &t)) return;
    const int64_t n0 = (int64_t)t.tn * T::BN;
    const int32_t m_left = t.end - t.row0 < T::BM ? t.end - t.row0 : T::BM;
    const int32_t n_left = (int32_t)(p.N - n0 < T::BN ? p.N - n0 : T::BN);
    T::run((lds_t *)smem_generic, row_operand(p, t, m_left), column_operand<OP>(p, t.e, n0, n_left),
           (int32_t)p.K, [&](int r, int c, const int (&v)[8]) {
               if (r < m_left && c < n_left) store_run<true, false>(p, (int64_t)t.row0 + r, n0 + c, v);
           });
}

template <int OP>
hipError_t launch_stream(GroupedArgs &a, hipStream_t s) {
    using T = StreamTile<OP>;
    a.tiles_n = (int32_t)((a.N + T::BN - 1) / T::BN);
    const int64_t blocks = (a.rows / T::BM + (a.E < a.rows ? a.E : a.rows)) * a.tiles_n;
    return launch_lds<grouped_stream_kernel<OP>>(blocks, T::THREADS, T::LDS_BYTES, s, a);
}

template <int OP, int BM, int BN, int WGM, int WGN, int SA, int SB>
hipError_t launch_tile(GroupedArgs &a, hipStream_t s) {
    using T = GroupedTile<OP, BM, BN, WGM, WGN, SA, SB>;
    a.tiles_n = (int32_t)((a.N + BN - 1) / BN);
    a.tiles_m = (int32_t)((a.K + BM - 1) / BM);
    int64_t blocks;
    if (OP == GEMM_GROUPED_TN) blocks = (((int64_t)a.tiles_m * a.tiles_n * a.parts + 7) / 8) * 8 * a.E;
    else blocks = (a.rows / BM + (a.E < a.rows ? a.E : a.rows)) * a.tiles_n;
    return launch_lds<grouped_tile_kernel<OP, BM, BN, WGM, WGN, SA, SB>>(blocks, T::THREADS, T::LDS_BYTES, s, a);
}

// Adds the parts of every weight gradient, in their order.
__global__ __launch_bounds__(256) void grouped_join_kernel(GroupedArgs p) {
    const int64_t runs = p.N / 8, all = (int64_t)p.E * p.K * runs;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / runs, n = i % runs * 8;
        if (p.accumulate) {          // nothing is added for an expert without rows, not even to -0
            int32_t lo, hi;
            group_rows(p, (int)(row / p.K), &lo, &hi);
            if (hi == lo) continue;
        }
        float x[8] = {};
#pragma unroll 4
        for (int s = 0; s < p.parts; ++s) {
            Raw<true> r;
            load8<true, true>(r, p.slots + ((int64_t)s * p.E * p.K + row) * p.N, (uint32_t)n, (uint32_t)p.N);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += raw_at(r, e);
        }
        int v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __float_as_int(x[e]);
        store_run<true, false>(p, row, n, v);
    }
}

template <int OP>
hipError_t launch_rows(GroupedArgs &a, hipStream_t s) {
    switch (rows_choice(a.rows, a.K, a.N, a.E)) {
    case kRows256: return launch_tile<OP, 256, 256, 2, 4, 2, 3>(a, s);
    case kRows128x256: return launch_tile<OP, 128, 256, 2, 4, 3, 3>(a, s);
    case kRows128: return launch_tile<OP, 128, 128, 2, 2, 2, 3>(a, s);
    case kRows128Deep: return launch_tile<OP, 128, 128, 2, 4, 4, 4>(a, s);
    case kRows64x128: return launch_tile<OP, 64, 128, 2, 2, 3, 3>(a, s);
    default: return launch_stream<OP>(a, s);
    }
}

// Weight gradients are many times the caches' size, so they are stored past them,
// and the caches keep the rows (repeated calls: 6001 rows, 32 experts of 2048 x 1792 in 32 bits:
// 111 us, 165 through them; 164 rows, 44 experts of 4040 x 2048: 223, 292).  Such
// stores have to cover whole lines (in runs of half a line: 589).  Rows that do
// not begin on a line break that at each tile's edge, which in 32 bits costs more
// than few rows per expert gain (20 experts of 1280 x 3576, 32 rows each 115 / 79,
// 64 rows 114 / 102, 128 rows 112 / 132; in bfloat16 56 / 50, 60 / 58, 74 / 70,
// but 34 experts of 3648 x 2248, 84 rows each 175 / 234).  Adding to C reads it in
// the epilogue: after a pass over 1 GB, 6001 rows, 32 experts of 2048 x 1792 in
// bfloat16 93 us, added to 192, in 32 bits 131 and 297; 16384 rows, 8 experts of 4096
// x 3584 429 and 507, 458 and 600.
bool stream_stores(const GroupedArgs &a) {
    return !a.out_f32 || (a.ldc % 32 == 0 && aligned(a.C, 128)) || a.rows / a.E >= 96;
}
hipError_t launch_tn(GroupedArgs &a, int max_parts, hipStream_t s) {
    const TnChoice c = tn_choice(a.rows, a.K, a.N, a.E);
    a.stream = stream_stores(a);
    if (c.large) return launch_tile<GEMM_GROUPED_TN, 256, 256, 2, 4, 2, 2>(a, s);
    a.parts = c.parts < max_parts ? c.parts : max_parts;    // (the slots hold max_parts)
    hipError_t e = launch_tile<GEMM_GROUPED_TN, 128, 128, 2, 2, 2, 3>(a, s);
    if (e != hipSuccess || a.parts == 1) return e;
    const int64_t blocks = ((int64_t)a.E * a.K * (a.N / 8) + 255) / 256;
    return launch(grouped_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), 256, 0, s, a);
}

template <int OP>
hipError_t launch_op(GroupedArgs &a, bool wide, int max_parts, hipStream_t s) {
    if (!wide) {
        a.tiles_n = (int32_t)((a.N + 63) / 64);
        a.tiles_m = (int32_t)((a.K + 63) / 64);
        const int64_t row_tiles = OP == GEMM_GROUPED_TN ? (int64_t)a.E * a.tiles_m
                                                        : a.rows / 64 + (a.E < a.rows ? a.E : a.rows);
        return launch(grouped_narrow_kernel<OP>, dim3((unsigned)(row_tiles * a.tiles_n)), 256, 0, s, a);
    }
    if constexpr (OP == GEMM_GROUPED_TN) return launch_tn(a, max_parts, s);
    else return launch_rows<OP>(a, s);
}

// Parts of any call of a plan: most for the most rows.
int most_parts(const gemm_grouped_desc_t &d) {
    if (d.op != GEMM_GROUPED_TN || d.N % 8 != 0 || d.K % 8 != 0) return 1;
    return tn_choice(d.M, d.K, d.N, d.E).parts;
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
    if (d.E > kMaxE || d.M > kMaxRows || d.N > INT32_MAX || d.K > INT32_MAX)
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
    int parts;           // most parts of a weight gradient
    float *slots;        // room for them, or null
    int64_t slot_bytes;
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
    hipError_t e = own(hipGetDevice(&p->device));
    if (e == hipSuccess) e = own(hipMalloc((void **)&p->err, 16));
    p->parts = most_parts(p->d);
    p->slot_bytes = p->parts > 1 ? p->parts * p->d.E * p->d.K * p->d.N * (int64_t)sizeof(float) : 0;
    if (e == hipSuccess && p->slot_bytes) e = own(hipMalloc((void **)&p->slots, p->slot_bytes));
    // a blocking copy: the word is zero before any later launch on any stream
    const int32_t zero[4] = {0, 0, 0, 0};
    if (e == hipSuccess) e = own(hipMemcpy(p->err, zero, 16, hipMemcpyHostToDevice));
    if (e != hipSuccess) {
        if (p->err) (void)own(hipFree(p->err));
        if (p->slots) (void)own(hipFree(p->slots));
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
    // arrays of no rows (A, and C or TN's B) need not have an address
    const bool tn = d.op == GEMM_GROUPED_TN, some = rows > 0;
    if ((!A && some) || (!B && (some || !tn)) || (!C && (some || tn)) || !offsets || !aligned(A, 2) ||
        !aligned(B, 2) || !aligned(offsets, 4) || !aligned(C, type_bytes(d.out_dtype)))
        return GEMM_RS_ERR_INVALID_ARG;
    if (rows == 0 && !tn) return GEMM_RS_OK;
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
    a.parts = 1;
    a.slots = p->slots;
    hipStream_t s = (hipStream_t)stream;
    const int64_t c_elems = d.out_dtype == GEMM_RS_F32 ? 4 : 8;
    const bool wide = d.N % 8 == 0 && d.K % 8 == 0 && d.lda % 8 == 0 && d.ldb % 8 == 0 &&
                      d.ldc % c_elems == 0 && aligned(A, 16) && aligned(B, 16) && aligned(C, 16);
    const hipError_t e = d.op == GEMM_GROUPED_NN   ? launch_op<GEMM_GROUPED_NN>(a, wide, p->parts, s)
                         : d.op == GEMM_GROUPED_NT ? launch_op<GEMM_GROUPED_NT>(a, wide, p->parts, s)
                                                   : launch_op<GEMM_GROUPED_TN>(a, wide, p->parts, s);
    return e == hipSuccess ? GEMM_RS_OK : GEMM_RS_ERR_HIP;
}

int gemm_grouped_status(gemm_grouped_plan_t p, void *stream, int32_t *detail) {
    if (!p || !on_device(p->device)) return GEMM_RS_ERR_INVALID_ARG;
    int32_t h[4] = {0, 0, 0, 0};
    hipError_t e = own(hipStreamSynchronize((hipStream_t)stream));
    if (e == hipSuccess) e = own(hipMemcpy(h, p->err, 16, hipMemcpyDeviceToHost));
    const int32_t zero[4] = {0, 0, 0, 0};
    if (e == hipSuccess && h[0] != 0) e = own(hipMemcpy(p->err, zero, 16, hipMemcpyHostToDevice));
    if (e != hipSuccess) return GEMM_RS_ERR_HIP;
    if (detail)
        for (int i = 0; i < 4; ++i) detail[i] = h[i];
    return h[0];
}

int gemm_grouped_query(gemm_grouped_plan_t p, gemm_grouped_info_t *info) {
    if (!p || !info) return GEMM_RS_ERR_INVALID_ARG;
    info->workspace_bytes = 16 + p->slot_bytes;
    return GEMM_RS_OK;
}

int gemm_grouped_destroy(gemm_grouped_plan_t p) {
    if (!p) return GEMM_RS_OK;
    int cur = -1;
    bool switched = false;
    if (own(hipGetDevice(&cur)) == hipSuccess && cur != p->device)
        switched = own(hipSetDevice(p->device)) == hipSuccess;
    // teardown is best effort: a failure here leaves nothing to undo
    (void)own(hipFree(p->err));
    if (p->slots) (void)own(hipFree(p->slots));
    if (switched) (void)own(hipSetDevice(cur));
    free(p);
    return GEMM_RS_OK;
}

}  // extern "C"
