// Matrix-pipe tile shared by the 8-bit product and the products grouped by
// expert: a BM x BN output tile per workgroup of WGM x WGN waves.
//
// Each step takes 128 bytes of the contraction from a row operand (one row
// of the contraction's 16-byte chunks per output row: 64 bfloat16, 128
// int8), or the 64 rows of a column operand (bfloat16, stored with the
// output axis contiguous).  Operands go from memory straight into rings of
// SA and SB stages in LDS, 16 bytes per lane; loads run SA - 1 and SB - 1 steps
// ahead.  Both kinds of LDS tile are XOR-swizzled in 16-byte chunks (by choosing the
// chunk that each lane fetches), so that fragment reads spread over the
// banks; a column operand's fragments come from transposing LDS reads.
//
// Everything outside an operand reads as zero: loads go through a buffer
// descriptor that ends with the operand's last valid byte of the step, and
// chunks past the end of the contraction are sent past the descriptor.  So no
// value in a gap or past an end, NaN or not, enters a sum, and rows and
// columns past the output are computed on zeros or on other tiles' values and
// never stored.
//
// Bounds.  A wave's WM x WN share of the output reads (WM + WN) * 128 bytes of
// LDS for WM * WN / 256 cycles of the matrix pipe in a step, so small shares
// are bound by LDS (128 x 128 tiles: 0.5 us a step, two thirds of it LDS reads
// and loads into LDS at 128 bytes a cycle), 128 x 64 ones (256 x 256 tiles) by
// the matrix pipe and, with every CU busy, by the board's power limit, which
// takes the clock to about 1.6 GHz: 8192 x 8192 x 3584 in int8 2040 TOP/s,
// 16384 rows over 8 experts of 4096 x 3584 in bfloat16 1100 TFLOP/s.  Reads and
// loads one by one behind the matrix operations instead of in batches: 1024 x
// 3584 x 8192 in int8 49 -> 39 us, 16384 rows 453 -> 438 us.
#pragma once

#include <type_traits>
#include <utility>

#include "ffn_internal.h"

namespace gemm_rs {
namespace ffn {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef short i16x8_t __attribute__((ext_vector_type(8)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) char lds_t;

#pragma clang diagnostic ignored "-Winline-asm"

// One 32 x 32 block: 16 bytes per lane of each operand (row lane % 32, the
// lane/32-th 16 bytes of the step), 16 deep in bfloat16, 32 deep in int8.
// The operands are swapped, so the block comes out transposed: a lane holds
// output row lane % 32, registers 4q..4q+3 its columns 8q + 4*(lane/32) + 0..3.
__device__ __forceinline__ f32x16_t mma(i32x4_t a, i32x4_t b, f32x16_t acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, b),
                                                   __builtin_bit_cast(bf16x8_t, a), acc, 0, 0, 0);
}
__device__ __forceinline__ i32x16_t mma(i32x4_t a, i32x4_t b, i32x16_t acc) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, acc, 0, 0, 0);
}
// One 16 x 16 block, 64 deep in int8: 16 bytes per lane of each operand (row
// lane % 16, the lane/16-th 16 bytes).  Swapped as above: a lane holds output
// row lane % 16, columns 4*(lane/16) + 0..3.
__device__ __forceinline__ i32x4_t mma16(i32x4_t a, i32x4_t b, i32x4_t acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, acc, 0, 0, 0);
}

// Raw buffer descriptor: 48-bit base, `bytes` records.  A load at or past
// `bytes` gives zeros (in LDS too, for a load to LDS).
__device__ __forceinline__ i32x4_t buffer_of(const void *base, uint32_t bytes) {
    const uint64_t p = (uint64_t)base;
    i32x4_t r;    // in scalar registers: the values are wave-uniform
    r[0] = __builtin_amdgcn_readfirstlane((int32_t)(uint32_t)p);
    r[1] = __builtin_amdgcn_readfirstlane((int32_t)((uint32_t)(p >> 32) & 0xffffu));
    r[2] = __builtin_amdgcn_readfirstlane((int32_t)bytes);
    r[3] = 0x00020000;
    return r;
}

// 16 bytes per lane into LDS: lane l's land at lds_base + 16 * l.  In asm so
// that the compiler does not wait for it before LDS reads of other stages;
// completion is tracked by wait_loads.
__device__ __forceinline__ void load_to_lds(i32x4_t rsrc, uint32_t voff, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :: "v"(voff), "s"(rsrc), "s"(lds_base) : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}
// Wait until at most `groups` (0..MAX) groups of PER loads are in flight.
template <int PER, int MAX>
__device__ __forceinline__ void wait_groups(int groups) {
    if constexpr (MAX > 0) {
        if (groups >= MAX) {
            wait_loads<MAX * PER>();
            return;
        }
        wait_groups<PER, MAX - 1>(groups);
    } else {
        wait_loads<0>();
    }
}

// Workgroup b of n, in an order that gives each XCD one run of the n tiles
// (the hardware deals workgroups out to the 8 XCDs in turn): neighbouring
// tiles share an operand, so they should share an L2.  A bijection of [0, n).
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t n) {
    const uint32_t x = b % 8, j = b / 8, q = n / 8, r = n % 8;
    return x * q + (x < r ? x : r) + j;
}

// One operand of a tile.  Row operand (COL false): `span` output rows from
// base, ld bytes apart, contraction along the row.  Column operand (COL
// true): contraction rows ld bytes apart, of which `span` bytes belong to
// the tile.  ld and base are multiples of 16; ld < 2^24, so that the
// offsets inside a step fit 32 bits.
struct Operand {
    const char *base;
    int64_t ld;
    int32_t span;

    // The same in scalar registers (the values are the same in every lane).
    __device__ __forceinline__ Operand scalar() const {
        const uint64_t p = (uint64_t)base;
        const uint32_t lo = __builtin_amdgcn_readfirstlane((int32_t)(uint32_t)p);
        const uint32_t hi = __builtin_amdgcn_readfirstlane((int32_t)(uint32_t)(p >> 32));
        return {(const char *)(((uint64_t)hi << 32) | lo),
                (int64_t)__builtin_amdgcn_readfirstlane((int32_t)ld), __builtin_amdgcn_readfirstlane(span)};
    }
};

template <class ACC, int BM_, int BN_, int WGM_, int WGN_, bool A_COL, bool B_COL, int SA, int SB = SA>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
    static constexpr int NW = WGM * WGN, THREADS = 64 * NW;
    static constexpr int WM = BM / WGM, WN = BN / WGN;
    static constexpr int FM = WM / 32, FN = WN / 32;
    static constexpr int KS = 4;                        // 32-byte slices of a step
    // Slices whose fragments are read together: at least 4 matrix operations
    // (of 32 cycles) to a batch, to cover the LDS latency of the next one.
    static constexpr int SL = FM * FN >= 4 ? 1 : FM * FN >= 2 ? 2 : 4;
    static constexpr int BATCHES = KS / SL;
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    static constexpr int LDS_BYTES = SA * A_BYTES + SB * B_BYTES;
    static_assert(SA >= 2 && (SB == SA || SB == SA + 1), "rings of A and B stages");
    // Loads of 1 KB per stage and operand, dealt out to all waves.
    static constexpr int AI = A_BYTES / 1024 / NW, BI = B_BYTES / 1024 / NW;
    static_assert(AI * NW * 1024 == A_BYTES && BI * NW * 1024 == B_BYTES, "whole loads per wave");
    static_assert(WM % 32 == 0 && WN % 32 == 0, "whole blocks per wave");
    static_assert(!A_COL || BM >= 128, "column swizzle needs 16 chunks per row");
    static_assert(!B_COL || BN >= 128, "column swizzle needs 16 chunks per row");
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
    static constexpr int A_READS = A_COL ? 2 * FM : FM, B_READS = B_COL ? 2 * FN : FN;

    // Row tiles: 8 chunks of 16 bytes per row, chunk c of row m at c ^ swz.
    static __device__ __forceinline__ int row_swz(int m) { return (m ^ (m >> 3)) & 7; }
    // Column tiles: chunk c of contraction row k at c ^ swz.
    static __device__ __forceinline__ int col_swz(int k) { return 4 * (k & 3); }

    ACC acc[FM][FN];

    // Load i of wave w covers 1 KB of an operand's tile, at (i * NW + w) * 1024:
    // this lane's chunk of it, and its offset from the window's base.
    template <bool COL, int B>
    static __device__ __forceinline__ int load_row(int i, int w, int lane) {
        return COL ? (i * NW + w) * (64 / (B / 8)) + lane / (B / 8) : (i * NW + w) * 8 + lane / 8;
    }
    template <bool COL, int B>
    static __device__ __forceinline__ int load_chunk(int i, int w, int lane) {
        const int r = load_row<COL, B>(i, w, lane);
        return COL ? (lane % (B / 8)) ^ col_swz(r) : (lane & 7) ^ row_swz(r);
    }
    template <bool COL, int B>
    static __device__ __forceinline__ uint32_t load_offset(const Operand &o, int i, int w, int lane) {
        return (uint32_t)load_row<COL, B>(i, w, lane) * (uint32_t)o.ld + (uint32_t)load_chunk<COL, B>(i, w, lane) * 16u;
    }
    // Descriptor of step kt's window, of which `left` (at most KE, none if
    // negative) elements, or rows of a column operand, are valid.  Rows past
    // the operand's lie past its end.
    template <bool COL, int ELEM>
    static __device__ __forceinline__ i32x4_t window(const Operand &o, int kt, int left) {
        const uint32_t bytes = COL ? (uint32_t)(left - 1) * (uint32_t)o.ld + (uint32_t)o.span
                                   : (uint32_t)(o.span - 1) * (uint32_t)o.ld + (uint32_t)(left * ELEM);
        return buffer_of(o.base + (COL ? (int64_t)kt * 64 * o.ld : (int64_t)kt * 128), left > 0 ? bytes : 0u);
    }

    // Steps of a contraction of k elements, ELEM bytes each.
    template <int ELEM> static __device__ __forceinline__ int steps_of(int32_t k) {
        return (int)(((uint32_t)k + 128 / ELEM - 1) / (128 / ELEM));
    }

    // acc = A . B over a contraction of `k` elements (of a column operand:
    // rows; ELEM bytes each in a row operand).
    template <int ELEM>
    __device__ __forceinline__ void run(lds_t *smem, const Operand &a_in, const Operand &b_in, int32_t k_in) {
        constexpr int KE = 128 / ELEM;
        static_assert(!(A_COL || B_COL) || KE == 64, "column operands are bfloat16");
        const Operand a = a_in.scalar(), b = b_in.scalar();
        const int k = __builtin_amdgcn_readfirstlane(k_in);
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WGN, wn = wave % WGN;
        const uint32_t smem_base = (uint32_t)(size_t)smem;
        const int KT = steps_of<ELEM>(k);

        constexpr int B_AT = SA * A_BYTES;               // B's stages follow A's
        uint32_t voff[AI + BI];
#pragma unroll
        for (int i = 0; i < AI; ++i) voff[i] = load_offset<A_COL, BM>(a, i, wave, lane);
#pragma unroll
        for (int i = 0; i < BI; ++i) voff[AI + i] = load_offset<B_COL, BN>(b, i, wave, lane);
        // row swizzles repeat every 64 rows, so a row operand's loads have at
        // most two chunk numbers; a column operand needs none (below)
        const int a_chunk[2] = {load_chunk<A_COL, BM>(0, wave, lane), load_chunk<A_COL, BM>(1, wave, lane)};
        const int b_chunk[2] = {load_chunk<B_COL, BN>(0, wave, lane), load_chunk<B_COL, BN>(1, wave, lane)};

        // A step's loads, one at a time.  Past the contraction's last step
        // they read nothing (and still count, so the waits are constants); in
        // its last step, chunks past the end of row operands are sent past
        // the descriptor (rows of column operands lie there already).
        struct Load {
            i32x4_t a, b;
            int a_chunks, b_chunks, a_to, b_to;
        };
        auto left_of = [&](int kt) __attribute__((always_inline)) {
            const int left = k - kt * KE;
            return left < KE ? left : KE;
        };
        auto begin_load = [&](int a_kt, int a_st, int b_kt, int b_st) __attribute__((always_inline)) {
            const int al = left_of(a_kt), bl = left_of(b_kt);
            return Load{window<A_COL, ELEM>(a, a_kt, al), window<B_COL, ELEM>(b, b_kt, bl),
                        al * ELEM / 16, bl * ELEM / 16, a_st, b_st};
        };
        auto load = [&](const Load &l, int i) __attribute__((always_inline)) {
            const bool isa = i < AI;
            const int j = isa ? i : i - AI;
            uint32_t v = voff[i];
            if (isa ? !A_COL : !B_COL)
                v = (isa ? a_chunk : b_chunk)[NW == 8 ? 0 : j & 1] < (isa ? l.a_chunks : l.b_chunks) ? v : 0xfffffff0u;
            load_to_lds(isa ? l.a : l.b, v,
                        smem_base + (isa ? l.a_to * A_BYTES : B_AT + l.b_to * B_BYTES) + (j * NW + wave) * 1024);
        };

        // LDS addresses of this lane's fragments: few registers, and constants
        // for the reads' immediate field.  Row operand: 16 bytes of row
        // lane % 32; block i lies i * 4096 further, with the row swizzle of
        // i's parity.  Column operand: two transposing reads of 4 x 16 blocks,
        // of which this lane addresses row te, columns 4 tq..4 tq + 3; slices and
        // halves lie whole rows further, blocks differ in the swizzled chunk.
        const int grp = lane >> 4, te = (lane & 15) >> 2, tq = lane & 3;
        lds_t *a_at[A_COL ? 1 : KS][A_COL ? FM : 2], *b_at[B_COL ? 1 : KS][B_COL ? FN : 2];
        auto col_at = [&](lds_t *tile, int x, int width) __attribute__((always_inline)) {
            const int n = x + 16 * (grp & 1) + 4 * tq, kk = 8 * (grp >> 1) + te;
            return tile + (kk * (width * 2) + (((n >> 3) ^ col_swz(kk)) << 4) + ((n & 7) << 1));
        };
        auto row_at = [&](lds_t *tile, int x, int odd, int ks) __attribute__((always_inline)) {
            const int m = x + (lane & 31), c = 2 * ks + (lane >> 5);
            return tile + (m * 128 + ((c ^ row_swz(m) ^ (4 * odd)) << 4));
        };
        if constexpr (A_COL) {
#pragma unroll
            for (int i = 0; i < FM; ++i) a_at[0][i] = col_at(smem, wm * WM + i * 32, BM);
        } else {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) a_at[ks][odd] = row_at(smem, wm * WM, odd, ks);
        }
        if constexpr (B_COL) {
#pragma unroll
            for (int j = 0; j < FN; ++j) b_at[0][j] = col_at(smem + B_AT, wn * WN + j * 32, BN);
        } else {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) b_at[ks][odd] = row_at(smem + B_AT, wn * WN, odd, ks);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = ACC{};

        auto col_read = [&](lds_t *at, int width) __attribute__((always_inline)) {
            typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
            const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)at);
            const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(at + 4 * width * 2));
            const i16x8_t both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(i32x4_t, both);
        };
        typedef __attribute__((address_space(3))) i32x4_t lds_i32x4;
        // Fragments are double-buffered in registers, SL slices of a step to a
        // batch: while the matrix pipe works on one batch the next one is read.
        constexpr int PER = FM + FN, READS = SL * PER, MM = SL * FM * FN, LOADS = AI + BI;
        i32x4_t af[2][SL][FM], bf[2][SL][FN];
        auto read = [&](int sa, int sb, int batch, int fb, int r) __attribute__((always_inline)) {
            const int s = r / PER, ks = batch * SL + s, i = r % PER, j = i - FM;
            if (i < FM) {
                if constexpr (A_COL) af[fb][s][i] = col_read(a_at[0][i] + sa * A_BYTES + ks * 16 * BM * 2, BM);
                else af[fb][s][i] = *(lds_i32x4 *)(a_at[ks][i & 1] + sa * A_BYTES + i * 4096);
            } else {
                if constexpr (B_COL) bf[fb][s][j] = col_read(b_at[0][j] + sb * B_BYTES + ks * 16 * BN * 2, BN);
                else bf[fb][s][j] = *(lds_i32x4 *)(b_at[ks][j & 1] + sb * B_BYTES + j * 4096);
            }
        };
        auto mma_one = [&](int fb, int m) __attribute__((always_inline)) {
            const int s = m / (FM * FN), i = m / FN % FM, j = m % FN;
            acc[i][j] = mma(af[fb][s][i], bf[fb][s][j], acc[i][j]);
        };
        auto mmas = [&](int fb) __attribute__((always_inline)) {
#pragma unroll
            for (int m = 0; m < MM; ++m) mma_one(fb, m);
        };
        // Step kt loads A's step kt + SA - 1 and B's step kt + SB - 1; the
        // first steps' loads, in the same order.
#pragma unroll
        for (int s = 1 - SB; s < 0; ++s) {
            const Load l = begin_load(s + SA - 1, s + SA - 1, s + SB - 1, s + SB - 1);
#pragma unroll
            for (int i = s + SA - 1 < 0 ? AI : 0; i < LOADS; ++i) load(l, i);
        }
        // Begins step kt: this wave's loads of it have landed (later steps' may
        // be in flight); behind the barrier every wave's have, and every wave
        // has read the stages that the loads of this step overwrite.
        auto arrive = [&](int kt, int sa, int sb) __attribute__((always_inline)) {
            wait_loads<(SA - 2) * LOADS + (SB > SA ? BI : 0)>();
            lds_only_barrier();
            int a_to = sa + SA - 1, b_to = sb + SB - 1;
            if (a_to >= SA) a_to -= SA;
            if (b_to >= SB) b_to -= SB;
            return begin_load(kt + SA - 1, a_to, kt + SB - 1, b_to);
        };
        // `parity`: of kt, a constant; `sa`, `sb`: kt % SA, kt % SB; `zeroth`:
        // kt is 0
        auto step = [&](int kt, auto a_stage, auto b_stage, auto parity, auto zeroth) __attribute__((always_inline)) {
            const int sa = a_stage, sb = b_stage;
            constexpr int P = decltype(parity)::value;
            constexpr int first = BATCHES == 1 ? P : 0;    // buffer of the step's first batch
            const Load l = arrive(kt, sa, sb);
            // A wave issues in order, and a read or a load waits its turn at
            // the LDS or the memory pipeline, so they go one by one behind
            // the matrix operations, which run meanwhile.
            if constexpr (decltype(zeroth)::value) {
#pragma unroll
                for (int r = 0; r < READS; ++r) read(sa, sb, 0, first, r);
#pragma unroll
                for (int i = 0; i < LOADS; ++i) load(l, i);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int batch = decltype(zeroth)::value ? 1 : 0; batch < BATCHES; ++batch) {
                const int into = (first + batch) & 1;
#pragma unroll
                for (int m = 0; m < MM; ++m) {
                    mma_one(1 - into, m);
#pragma unroll
                    for (int r = m * READS / MM; r < (m + 1) * READS / MM; ++r) read(sa, sb, batch, into, r);
                    if (batch == 0)
#pragma unroll
                        for (int i = m * LOADS / MM; i < (m + 1) * LOADS / MM; ++i) load(l, i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        using Even = std::integral_constant<int, 0>;
        using Odd = std::integral_constant<int, 1>;
        // two steps per turn, so that fragment buffers, and stages of a ring
        // of two (which go into the LDS reads' immediate field), are constants
        using No = std::false_type;
        int kt = 0, sa = 0, sb = 0;
        auto next = [&]() __attribute__((always_inline)) {
            ++kt;
            if (++sa == SA) sa = 0;
            if (++sb == SB) sb = 0;
        };
        // a wave whose rows or columns all lie past the output's only loads
        const int rows = A_COL ? a.span / 2 : a.span, cols = B_COL ? b.span / 2 : b.span;
        if (wm * WM >= rows || wn * WN >= cols) {
            while (kt < KT) {
                const Load l = arrive(kt, sa, sb);
#pragma unroll
                for (int i = 0; i < LOADS; ++i) load(l, i);
                next();
            }
            return;
        }
        auto turn = [&](auto parity, auto zeroth) __attribute__((always_inline)) {
            if constexpr (SB == 2) step(kt, parity, parity, parity, zeroth);
            else if constexpr (SA == 2) step(kt, parity, sb, parity, zeroth);
            else step(kt, sa, sb, parity, zeroth);
            next();
        };
        if (KT > 0) turn(Even{}, std::true_type{});
        while (kt + 1 < KT) {
            turn(Odd{}, No{});
            turn(Even{}, No{});
        }
        if (kt < KT) turn(Odd{}, No{});
        if (KT > 0) {
            if (BATCHES > 1 || KT % 2 == 0) mmas(1);
            else mmas(0);
        }
    }

    // Hands the tile out as f(row, c0, c1, v[8]): columns c0..c0 + 3 and c1..c1 + 3
    // of a row, every column once, whole rows by neighbouring lanes.  c1 is c0 + 4,
    // or with SPLIT (for 32-bit outputs) c0 + BN / 2, so that one 16-byte store of
    // the lanes of a row covers a run of it either way.  Accumulators pass through LDS one 32-row block
    // row of every wave at a time: the direct layout would store 8 bytes per
    // row and instruction.  16-byte chunk c of a staged row r sits at
    // c ^ (r % 16).
    template <bool SPLIT, class F>
    __device__ __forceinline__ void store(lds_t *smem, F f) const {
        constexpr int SROWS = WGM * 32, ROW = BN * 4, SBYTES = SROWS * ROW;
        constexpr bool TWICE = 2 * SBYTES <= LDS_BYTES;   // alternate between two halves
        static_assert(SBYTES <= LDS_BYTES, "a stripe fits");
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WGN, wn = wave % WGN;
        typedef __attribute__((address_space(3))) i32x4_t lds_i32x4;
        wait_loads<0>();                                  // the empty loads past the last step
        lds_only_barrier();                               // every wave is done with the stages
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            lds_t *const s = smem + (TWICE ? (i & 1) * SBYTES : 0);
            if (!TWICE && i > 0) lds_only_barrier();
            {
                const int rr = wm * 32 + (lane & 31);
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = (wn * WN + j * 32 + 8 * q) / 4 + (lane >> 5);
                        i32x4_t v;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const auto x = acc[i][j][4 * q + e];
                            v[e] = __builtin_bit_cast(int32_t, x);
                        }
                        *(lds_i32x4 *)(s + rr * ROW + ((c ^ (rr & 15)) << 4)) = v;
                    }
            }
            lds_only_barrier();
            constexpr int LPR = BN / 8;
#pragma unroll
            for (int u = 0; u < SROWS * LPR; u += THREADS) {
                const int rr = (u + tid) / LPR;
                const int c = SPLIT ? tid % LPR : (tid % LPR) * 2, d = SPLIT ? c + LPR : c + 1;
                const i32x4_t lo = *(lds_i32x4 *)(s + rr * ROW + ((c ^ (rr & 15)) << 4));
                const i32x4_t hi = *(lds_i32x4 *)(s + rr * ROW + ((d ^ (rr & 15)) << 4));
                const int v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                f((rr >> 5) * WM + i * 32 + (rr & 31), c * 4, d * 4, v);
            }
        }
    }
};

}  // namespace ffn
}  // namespace gemm_rs
