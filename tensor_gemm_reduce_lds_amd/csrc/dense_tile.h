// Dense products of more than a few rows: matrix-pipe tiles, and the kernel for
// operands that they do not take.
#pragma once

#include "dense.h"

namespace gemm_rs {
namespace ffn {

// ---- matrix-pipe tiles ---------------------------------------------------------
template <TileKind KIND, bool A_COL, bool B_COL, int BM, int BN, int WGM, int WGN, int SA, int SB>
using DenseTile = Tile<f32x16_t, BM, BN, WGM, WGN, A_COL, B_COL, SA, SB, KIND>;

// A tile's place in a launch.
struct TileAt {
    int which, part;          // of several gradients; of the contraction
    int64_t index;            // among all tiles
    int64_t m0, n0;
    int32_t m_left;
};
// Workgroup b's tile.  Row tiles in groups of 8, a group column by column, so that
// the tiles that run together read few rows of A and columns of B.
template <class T>
__device__ __forceinline__ TileAt tile_at(const DenseArgs &p, uint32_t b) {
    const uint32_t tiles = (uint32_t)p.tiles_m * (uint32_t)p.tiles_n, unit = b / tiles, t = b - unit * tiles;
    const uint32_t group = t / (8 * (uint32_t)p.tiles_n), in = t - group * 8 * (uint32_t)p.tiles_n;
    const uint32_t tall = (uint32_t)p.tiles_m - group * 8 < 8 ? (uint32_t)p.tiles_m - group * 8 : 8;
    TileAt at;
    at.part = (int)(unit / (uint32_t)p.count);
    at.which = (int)(unit % (uint32_t)p.count);
    at.index = (int64_t)at.which * tiles + t;
    at.m0 = (int64_t)(group * 8 + in % tall) * T::BM;
    at.n0 = (int64_t)(in / tall) * T::BW;
    at.m_left = (int32_t)(p.rows - at.m0 < T::BM ? p.rows - at.m0 : T::BM);
    return at;
}

// Parts of a contraction: each part's workgroups store their sums, turn by turn as
// their threads have them, and a second kernel's threads add those of the same place,
// in the order of the parts, and finish them.  (In the last workgroup to arrive at a
// tile instead, with sums stored and loaded past the L2s, the sum is as long as the
// kernel it saves: 64 rows, 4096 x 1792 gated 17.2 us against 15.1, 3584 x 8192 21.4
// against 20.5; 16 rows 17.0 against 18.0.)
template <class T>
__device__ __forceinline__ float *slot_of(const DenseArgs &p, const TileAt &t, int part, int turn) {
    return p.slots + ((t.index * p.parts + part) * (T::BM * T::BN) + ((int64_t)turn * T::THREADS + threadIdx.x) * 4);
}
template <class T, int NV>
__device__ __forceinline__ void put_part(const DenseArgs &p, const TileAt &t, int turn, const int (&v)[NV]) {
#pragma unroll
    for (int h = 0; h < NV / 4; ++h)
        *(i32x4_t *)slot_of<T>(p, t, t.part, turn * (NV / 4) + h) = i32x4_t{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
}
template <class T, int NV>
__device__ __forceinline__ void sum_parts(const DenseArgs &p, const TileAt &t, int turn, int (&v)[NV]) {
    float z[NV] = {};
#pragma unroll 8
    for (int s = 0; s < p.parts; ++s)
#pragma unroll
        for (int h = 0; h < NV / 4; ++h) {
            const f32x4_t w = *(const f32x4_t *)slot_of<T>(p, t, s, turn * (NV / 4) + h);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[4 * h + e] += w[e];
        }
#pragma unroll
    for (int e = 0; e < NV; ++e) v[e] = __float_as_int(z[e]);
}

// What finishes a tile's values as a thread gets them.  RES: residuals are fetched
// ahead, those of all stripes at once, but of floats, for which few registers are left,
// of two, and each of the others when its place is free (8192 x 8192 x 3584 in floats
// with bias and residual 512 us; a stripe at a time 524, of three 549).  Beside the 128
// accumulators of a 256 x 256 tile's thread they leave too few registers in the
// epilogue, which spills 19 to 21 of them (48 and 56 bytes of scratch a lane), and 49
// (92 bytes) in the weight gradients, where all forms of output, added to or not, are
// one kernel; the loop over the contraction spills none.
template <class T, bool F32, bool STREAM, bool RES>
struct FinishOne {
    static constexpr auto ORDER = F32 ? T::kSplit : T::kRun8;
    static constexpr int NV = 8, U = T::template turns<ORDER>(), N = F32 || RES ? 1 : U, APART = F32 ? T::BN / 2 : 4;
    static constexpr int HELD = !RES ? 1 : F32 && T::FM > 2 ? 2 : T::FM;
    static constexpr bool LOOP = !RES;
    const DenseArgs &p;
    const TileAt &t;
    const Columns at;
    const int lane_row;
    float b[8];
    Raw<F32> res[HELD][U];

    __device__ __forceinline__ FinishOne(const DenseArgs &p_, const TileAt &t_)
        : p(p_), t(t_), at(t_.n0 + T::template column<ORDER>(), t_.n0 + T::template column<ORDER>() + APART, p_.N),
          lane_row(T::template thread_row<ORDER>()) {
        float lo[4], hi[4];
        bias_at(p.bias[0], p.bias_f32, at.c, p.N, lo);
        bias_at(p.bias[0], p.bias_f32, at.d, p.N, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            b[e] = lo[e];
            b[4 + e] = hi[e];
        }
    }
    __device__ __forceinline__ bool inside(int i, int u) const { return T::template row_of_turn<ORDER>(i, u) + lane_row < t.m_left; }
    __device__ __forceinline__ RowAt row(int i, int u) const { return {t.m0 + T::template row_of_turn<ORDER>(i, u), (uint32_t)lane_row}; }
    __device__ __forceinline__ void fetch(int i, int u) {
        // (rows past the output's last one stand for earlier ones)
        const int turn = T::template row_of_turn<ORDER>(i, u), r = turn < t.m_left ? turn : t.m_left - 1;
        const int most = t.m_left - 1 - r;
        fetch_residual<F32>(p, res[i % HELD][u], {t.m0 + r, (uint32_t)(lane_row < most ? lane_row : most)}, at);
    }
    __device__ __forceinline__ void before() {
        if constexpr (RES)
#pragma unroll
            for (int i = 0; i < HELD; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u) fetch(i, u);
    }
    // `n` of a stripe's turns from `first` on, their residuals from r on
    template <int n>
    __device__ __forceinline__ void finish(int i, int first, const int (&v)[n][8], const Raw<F32> *r) const {
        float z[n * 8];
#pragma unroll
        for (int u = 0; u < n; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[u * 8 + e] = __int_as_float(v[u][e]) + b[e];
        finish_one<F32, STREAM, n>(p, t.which, at, z, r, [&](int u) { return inside(i, first + u); }, [&](int u) { return row(i, first + u); });
    }
    template <int AT>
    __device__ __forceinline__ void operator()(int i, std::integral_constant<int, AT>, int first, const int (&v)[N][8]) {
        finish(i, first, v, RES ? res[AT % HELD] + first : nullptr);
        if constexpr (RES && AT + HELD < T::FM)      // (into the places that are done)
#pragma unroll
            for (int u = 0; u < N; ++u) fetch(AT + HELD, first + u);
    }
    __device__ __forceinline__ void one(int i, int u, const int (&v)[1][8]) const {
        Raw<F32> r[1] = {};
        if (p.R) fetch_residual<F32>(p, r[0], row(i, u), at);
        finish(i, u, v, r);
    }
};
template <class T, bool STREAM>
struct FinishPair {
    static constexpr auto ORDER = T::kTwoRuns;
    static constexpr int NV = 16, U = T::template turns<ORDER>(), N = U;
    static constexpr bool LOOP = true;
    const DenseArgs &p;
    const TileAt &t;
    const Columns at;
    const int lane_row;
    float b0[8], b1[8];

    __device__ __forceinline__ FinishPair(const DenseArgs &p_, const TileAt &t_)
        : p(p_), t(t_), at(t_.n0 + T::template column<ORDER>(), t_.n0 + T::template column<ORDER>() + 4, p_.N),
          lane_row(T::template thread_row<ORDER>()) {
        bias_at(p.bias[0], p.bias_f32, at.c, p.N, b0);
        bias_at(p.bias[1], p.bias_f32, at.c, p.N, b1);
    }
    __device__ __forceinline__ bool inside(int i, int u) const { return T::template row_of_turn<ORDER>(i, u) + lane_row < t.m_left; }
    __device__ __forceinline__ void before() {}
    template <int n>
    __device__ __forceinline__ void finish(int i, int first, const int (&v)[n][16]) const {
        float z0[n * 8], z1[n * 8];
#pragma unroll
        for (int u = 0; u < n; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z0[u * 8 + e] = __int_as_float(v[u][e]) + b0[e];
                z1[u * 8 + e] = __int_as_float(v[u][8 + e]) + b1[e];
            }
        finish_pair<STREAM, n>(p, at, z0, z1, [&](int u) { return inside(i, first + u); },
                               [&](int u) { return RowAt{t.m0 + T::template row_of_turn<ORDER>(i, first + u), (uint32_t)lane_row}; });
    }
    template <int P>
    __device__ __forceinline__ void operator()(int i, std::integral_constant<int, P>, int first, const int (&v)[N][16]) const { finish(i, first, v); }
    __device__ __forceinline__ void one(int i, int u, const int (&v)[1][16]) const { finish(i, u, v); }
};

// f(FINISH) for the type of finish that a launch's outputs take; `ahead`: with
// residuals fetched ahead, if there are any.
template <TileKind KIND, bool A_COL, class T, class F>
__device__ __forceinline__ void with_finish(const DenseArgs &p, const TileAt &t, bool ahead, F f) {
    auto of = [&](auto f32, auto stream) __attribute__((always_inline)) {
        if constexpr (KIND == kPair) {
            FinishPair<T, decltype(stream)::value> finish(p, t);
            f(finish);
        } else {
            constexpr bool F32 = decltype(f32)::value, STREAM = decltype(stream)::value;
            DenseArgs q = p;
            if (A_COL && p.add) q.R = t.which ? p.D[1] : p.D[0];
            if (KIND == kOne && q.R && ahead) {
                FinishOne<T, F32, STREAM, KIND == kOne> finish(q, t);
                f(finish);
            } else {
                FinishOne<T, F32, STREAM, false> finish(q, t);
                f(finish);
            }
        }
    };
    auto type = [&](auto f32) __attribute__((always_inline)) {
        if (A_COL && p.stream) of(f32, std::integral_constant<bool, A_COL>{});
        else of(f32, std::false_type{});
    };
    if (KIND != kPair && p.out_f32) type(std::true_type{});
    else type(std::false_type{});
}

// The geometry of a tile, whatever its operands and stages are.
template <int BM, int BN, int WGM, int WGN, bool PAIR>
using JoinTile = Tile<f32x16_t, BM, BN, WGM, WGN, false, false, 2, 2, PAIR ? kPair : kOne>;

template <TileKind KIND, bool A_COL, bool B_COL, int BM, int BN, int WGM, int WGN, int SA, int SB>
__global__ __launch_bounds__(64 * WGM * WGN) void dense_tile_kernel(DenseArgs p) {
    using T = DenseTile<KIND, A_COL, B_COL, BM, BN, WGM, WGN, SA, SB>;
    constexpr int BW = T::BW;
    extern __shared__ __attribute__((aligned(1024))) char smem_generic[];
    lds_t *smem = (lds_t *)smem_generic;
    // Each XCD takes one run of the tiles: part by part, gradient by gradient.
    const TileAt t = tile_at<T>(p, xcd_run(blockIdx.x, gridDim.x));
    const int32_t n_left = (int32_t)(p.N - t.n0 < BW ? p.N - t.n0 : BW);
    const uint32_t steps = (uint32_t)((p.K + 63) / 64);
    const int64_t k0 = (int64_t)((uint64_t)t.part * steps / p.parts) * 64;
    const int64_t k1 = t.part + 1 == p.parts ? p.K : (int64_t)((uint64_t)(t.part + 1) * steps / p.parts) * 64;
    auto a_at = [&](const uint16_t *q) { return (const char *)(q + (A_COL ? k0 * p.lda + t.m0 : t.m0 * p.lda + k0)); };
    auto b_at = [&](const uint16_t *q) { return (const char *)(q + (B_COL ? k0 * p.ldb + t.n0 : t.n0 * p.ldb + k0)); };
    // (rows of column operands are whole runs of 8: N is, or they are padded copies)
    const Operand a = {a_at(t.which ? p.A[1] : p.A[0]), p.lda * 2, A_COL ? (t.m_left + 7) / 8 * 16 : t.m_left, KIND == kParts ? a_at(p.A[1]) : nullptr};
    const Operand o = {b_at(t.which ? p.B[1] : p.B[0]), p.ldb * 2, B_COL ? (n_left + 7) / 8 * 16 : n_left, KIND != kOne ? b_at(p.B[1]) : nullptr};
    T tile;
    tile.template run<2>(smem, a, o, (int32_t)(k1 - k0));
    with_finish<KIND, A_COL, T>(p, t, p.parts == 1, [&](auto &finish) __attribute__((always_inline)) {
        using F = std::remove_reference_t<decltype(finish)>;
        if (F::LOOP && p.parts > 1)
            tile.template hand_out<F::ORDER, F::N, true>(smem, [] {}, [&](int i, auto, int first, const int (&v)[F::N][F::NV]) __attribute__((always_inline)) {
#pragma unroll
                for (int u = 0; u < F::N; ++u)
                    if (finish.inside(i, first + u)) put_part<T, F::NV>(p, t, i * F::U + first + u, v[u]);
            });
        else
            tile.template hand_out<F::ORDER, F::N, F::LOOP>(smem, [&]() __attribute__((always_inline)) { finish.before(); },
                                                            [&](int i, auto which, int first, const int (&v)[F::N][F::NV]) __attribute__((always_inline)) { finish(i, which, first, v); });
    });
}

// A workgroup for each turn of each tile, with the tile's threads.
template <TileKind KIND, bool A_COL, class T>
__global__ __launch_bounds__(T::THREADS) void dense_join_kernel(DenseArgs p) {
    const TileAt t = tile_at<T>(p, blockIdx.x);
    with_finish<KIND, A_COL, T>(p, t, false, [&](auto &finish) __attribute__((always_inline)) {
        using F = std::remove_reference_t<decltype(finish)>;
        const int turn = (int)blockIdx.y, i = turn / F::U, u = turn % F::U;
        if (!finish.inside(i, u)) return;
        int v[1][F::NV];
        sum_parts<T, F::NV>(p, t, turn, v[0]);
        finish.one(i, u, v);
    });
}

// ---- any size, stride and alignment --------------------------------------------
// For operands that the others do not take: 64 x 64 outputs (of each array of a
// pair) per workgroup, 32 x 32 per wave, 64 of the contraction at a time, loaded
// through registers (16 bytes at any element address, zeros outside the operand)
// two steps ahead, and written to the other of two LDS buffers one step ahead.
__device__ __forceinline__ int dense_row_swz(int r) { return (r ^ (r >> 3)) & 7; }
__device__ __forceinline__ int dense_col_swz(int r) { return 4 * ((r >> 1) & 1); }
// A fragment of a 64 x 128-byte LDS tile: 16 bytes of row m + lane % 32 of slice
// ks, or of a column operand by two transposing reads (rows r and r + 4 have the
// same swizzle).
template <bool COL>
__device__ __forceinline__ i32x4_t dense_fragment(lds_t *tile, int m, int ks) {
    typedef __attribute__((address_space(3))) i32x4_t lds_i32x4;
    typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
    const int lane = threadIdx.x & 63;
    if constexpr (COL) {
        const int grp = lane >> 4, te = (lane & 15) >> 2, tq = lane & 3;
        const int r = ks * 16 + 8 * (grp >> 1) + te, x = m + 16 * (grp & 1) + 4 * tq;
        lds_t *const q = tile + r * 128 + (((x >> 3) ^ dense_col_swz(r)) << 4) + ((x & 7) << 1);
        const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)q);
        const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(q + 4 * 128));
        return __builtin_bit_cast(i32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        const int r = m + (lane & 31);
        return *(lds_i32x4 *)(tile + r * 128 + (((2 * ks + (lane >> 5)) ^ dense_row_swz(r)) << 4));
    }
}

template <TileKind KIND, bool A_COL, bool B_COL>
__global__ __launch_bounds__(256) void dense_narrow_kernel(DenseArgs p) {
    constexpr int ARRAYS = KIND == kPair ? 2 : 1, STAGE = (1 + ARRAYS) * 8192;
    __shared__ __attribute__((aligned(1024))) char smem_generic[2 * STAGE];
    lds_t *const smem = (lds_t *)smem_generic;        // [buffer][A, B, B']
    typedef __attribute__((address_space(3))) u32x4_t lds_u32x4;
    typedef __attribute__((address_space(3))) f32x4_t lds_f32x4;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t tiles = (uint32_t)p.tiles_m * (uint32_t)p.tiles_n;
    const uint32_t b = xcd_run(blockIdx.x, gridDim.x), t = b % tiles;
    const int which = (int)(b / tiles);
    const int64_t m0 = (int64_t)(t % (uint32_t)p.tiles_m) * 64, n0 = (int64_t)(t / (uint32_t)p.tiles_m) * 64;
    // this thread's chunks: number tid % 8 of rows tid / 8 and 32 further
    const int chunk = tid & 7;
    const int64_t steps = (p.K + 63) / 64, all = KIND == kParts ? 2 * steps : steps;
    Raw<false> ra[2][2], rb[2][ARRAYS][2];            // of two steps
    auto take = [&](Raw<false> &r, const uint16_t *at, int64_t ld, int64_t row, int64_t rows, int64_t from, int64_t upto) __attribute__((always_inline)) {
        r = Raw<false>{};
        if (row < rows && from + chunk * 8 < upto)
            fetch8<false, false>(r, at + row * ld, (uint32_t)from + chunk * 8, (uint32_t)upto);
    };
    auto k_of = [&](int64_t step) { return (KIND == kParts && step >= steps ? step - steps : step) * 64; };
    auto fetch = [&](int set, int64_t step) __attribute__((always_inline)) {
        const int64_t k0 = k_of(step), k_len = step < all ? p.K : 0;      // (nothing past the end)
        const int second = KIND == kParts ? step >= steps : which;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (tid >> 3) + 32 * i;
            const uint16_t *const A = second ? p.A[1] : p.A[0];
            if constexpr (A_COL) take(ra[set][i], A, p.lda, k0 + r, k_len, m0, p.rows);
            else take(ra[set][i], A, p.lda, m0 + r, p.rows, k0, k_len);
#pragma unroll
            for (int a = 0; a < ARRAYS; ++a) {
                const uint16_t *const B = second || a ? p.B[1] : p.B[0];
                if constexpr (B_COL) take(rb[set][a][i], B, p.ldb, k0 + r, k_len, n0, p.N);
                else take(rb[set][a][i], B, p.ldb, n0 + r, p.N, k0, k_len);
            }
        }
    };
    // (rows past an operand's hold zeros, which the shift leaves)
    auto put = [&](int set, int64_t step) __attribute__((always_inline)) {
        const int64_t k0 = k_of(step), k_len = step < all ? p.K : 0;
        const uint32_t a_from = (uint32_t)(A_COL ? m0 : k0) + chunk * 8, b_from = (uint32_t)(B_COL ? n0 : k0) + chunk * 8;
        const uint32_t a_upto = (uint32_t)(A_COL ? p.rows : k_len), b_upto = (uint32_t)(B_COL ? p.N : k_len);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (tid >> 3) + 32 * i;
            lds_t *const at = smem + set * STAGE + r * 128;
            settle8<false, false>(ra[set][i], a_from, a_upto);
            *(lds_u32x4 *)(at + ((chunk ^ (A_COL ? dense_col_swz(r) : dense_row_swz(r))) << 4)) = ra[set][i].a;
#pragma unroll
            for (int a = 0; a < ARRAYS; ++a) {
                settle8<false, false>(rb[set][a][i], b_from, b_upto);
                *(lds_u32x4 *)(at + (1 + a) * 8192 + ((chunk ^ (B_COL ? dense_col_swz(r) : dense_row_swz(r))) << 4)) = rb[set][a][i].a;
            }
        }
    };
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    f32x16_t acc[ARRAYS] = {};
    fetch(0, 0);
    fetch(1, 1);
    put(0, 0);
    lds_only_barrier();
    auto step = [&](int now, int64_t s) __attribute__((always_inline)) {
        fetch(now, s + 2);
        lds_t *const at = smem + now * STAGE;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const i32x4_t af = dense_fragment<A_COL>(at, wm, ks);
#pragma unroll
            for (int a = 0; a < ARRAYS; ++a) acc[a] = mma(af, dense_fragment<B_COL>(at + (1 + a) * 8192, wn, ks), acc[a]);
        }
        put(now ^ 1, s + 1);
        lds_only_barrier();
    };
    for (int64_t s = 0; s < all; s += 2) {
        step(0, s);
        if (s + 1 < all) step(1, s + 1);
    }
    // through LDS, so that runs of 8 columns are finished together
    const int m = wm + (lane & 31);
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f32x4_t v = {acc[a][4 * q], acc[a][4 * q + 1], acc[a][4 * q + 2], acc[a][4 * q + 3]};
            *(lds_f32x4 *)(smem + a * 16384 + m * 256 + (((wn / 4 + 2 * q + (lane >> 5)) ^ (m & 15)) << 4)) = v;
        }
    lds_only_barrier();
    DenseArgs o = p;
    if (A_COL && p.add) o.R = which ? p.D[1] : p.D[0];
    const Columns at(n0 + chunk * 8, n0 + chunk * 8 + 4, p.N);
    float bias[ARRAYS][8];
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a) bias_at(p.bias[a], p.bias_f32, at.c, p.N, bias[a]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = (tid >> 3) + 32 * i;
        if (m0 + r >= p.rows || at.c_left == 0) continue;
        float z[ARRAYS][8];
#pragma unroll
        for (int a = 0; a < ARRAYS; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4_t x = *(lds_f32x4 *)(smem + a * 16384 + r * 256 + (((2 * chunk + h) ^ (r & 15)) << 4));
#pragma unroll
                for (int u = 0; u < 4; ++u) z[a][4 * h + u] = x[u] + bias[a][4 * h + u];
            }
        const RowAt row = {m0 + r, 0};
        auto inside = [](int) { return true; };
        auto row_at = [&](int) { return row; };
        if constexpr (KIND == kPair) {
            finish_pair<false, 1>(o, at, z[0], z[1], inside, row_at);
        } else if (p.out_f32) {
            Raw<true> res[1] = {};
            if (o.R) fetch_short_residual<true>(o, res[0], row, at);
            finish_one<true, false, 1>(o, which, at, z[0], res, inside, row_at);
        } else {
            Raw<false> res[1] = {};
            if (o.R) fetch_short_residual<false>(o, res[0], row, at);
            finish_one<false, false, 1>(o, which, at, z[0], res, inside, row_at);
        }
    }
}

// ---- launches ------------------------------------------------------------------
// `parts` as far as the plan's memory has room for them.
template <TileKind KIND, bool A_COL, bool B_COL, int BM, int BN, int WGM, int WGN, int SA, int SB>
hipError_t launch_dense_tile(DenseArgs &a, int parts, int64_t slot_bytes, hipStream_t s) {
    using T = DenseTile<KIND, A_COL, B_COL, BM, BN, WGM, WGN, SA, SB>;
    a.tiles_m = (int32_t)((a.rows + BM - 1) / BM);
    a.tiles_n = (int32_t)((a.N + T::BW - 1) / T::BW);
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n * a.count, room = slot_bytes / (tiles * BM * BN * (int64_t)sizeof(float));
    a.parts = room < 2 ? 1 : parts < room ? parts : (int)room;
    const hipError_t e = launch_lds<dense_tile_kernel<KIND, A_COL, B_COL, BM, BN, WGM, WGN, SA, SB>>(tiles * a.parts, T::THREADS, T::LDS_BYTES, s, a);
    if (e != hipSuccess || a.parts == 1) return e;
    using J = JoinTile<BM, BN, WGM, WGN, KIND == kPair>;
    const int turns = T::FM * (KIND == kPair ? J::template turns<J::kTwoRuns>() : a.out_f32 ? J::template turns<J::kSplit>() : J::template turns<J::kRun8>());
    return launch(dense_join_kernel<KIND, A_COL, J>, dim3((unsigned)tiles, (unsigned)turns), J::THREADS, 0, s, a);
}

template <TileKind KIND, bool A_COL, bool B_COL>
hipError_t launch_dense_narrow(DenseArgs &a, hipStream_t s) {
    a.tiles_m = (int32_t)((a.rows + 63) / 64);
    a.tiles_n = (int32_t)((a.N + 63) / 64);
    return launch(dense_narrow_kernel<KIND, A_COL, B_COL>, dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n * a.count)), 256, 0, s, a);
}

template <TileKind KIND, bool COL>
hipError_t launch_dense_form(DenseArgs &a, bool direct, int64_t slot_bytes, hipStream_t s) {
    a.count = 1;
    if constexpr (!COL)
        if (a.rows <= kFewRows && (direct || a.K >= 8)) return launch_dense_rows<KIND>(a, direct, s);
    // (the tiles fetch residuals in runs of 8)
    if (!direct || (a.R && a.N < 8)) return launch_dense_narrow<KIND, false, COL>(a, s);
    const DenseWay way = dense_choice(a.rows, a.N, a.K * (KIND == kParts ? 2 : 1), KIND == kPair ? 2 : 1, COL);
    const int n = way.parts;
    const int64_t b = slot_bytes;
    switch (way.kernel) {
    case kDense256: return launch_dense_tile<KIND, false, COL, 256, 256, 2, 4, 2, 3>(a, n, b, s);
    case kDense128x256: return launch_dense_tile<KIND, false, COL, 128, 256, 2, 4, 3, 3>(a, n, b, s);
    case kDense128: return launch_dense_tile<KIND, false, COL, 128, 128, 2, 2, 2, 3>(a, n, b, s);
    case kDense128Deep: return launch_dense_tile<KIND, false, COL, 128, 128, 2, 4, 4, 4>(a, n, b, s);
    default: return launch_dense_tile<KIND, false, COL, 64, 128, 2, 2, 3, 3>(a, n, b, s);
    }
}

// All rows, in as many launches as they take.
template <TileKind KIND>
hipError_t launch_dense(DenseArgs &all, bool col, bool direct, int64_t slot_bytes, hipStream_t s) {
    const int64_t most = rows_of_launch(all.N);
    for (int64_t r = 0; r < all.rows; r += most) {
        DenseArgs a = all;
        auto below = [r](const void *p, int64_t ld, int elem) { return p ? (char *)p + r * ld * elem : nullptr; };
        a.rows = all.rows - r < most ? all.rows - r : most;
        for (const uint16_t *&A : a.A) A = (const uint16_t *)below(A, a.lda, 2);
        a.R = below(a.R, a.ldr, a.out_f32 ? 4 : 2);
        a.D[0] = below(a.D[0], a.ldd, a.out_f32 ? 4 : 2);
        for (void *&Z : a.Z) Z = below(Z, a.ldz, a.z_f32 ? 4 : 2);
        const hipError_t e = col ? launch_dense_form<KIND, true>(a, direct, slot_bytes, s) : launch_dense_form<KIND, false>(a, direct, slot_bytes, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace ffn
}  // namespace gemm_rs
