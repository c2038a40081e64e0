// Matrix-pipe tile shared by the 8-bit product and the products grouped by
// expert: a BM x BN output tile per workgroup of WGM x WGN waves.
//
// Each step takes 128 bytes of the contraction from a row operand (one row
// of the contraction's 16-byte chunks per output row: 64 bfloat16, 128
// int8), or the 64 rows of a column operand (bfloat16, stored with the
// output axis contiguous).  Operands go from memory straight into a ring of
// STAGES stages in LDS, 16 bytes per lane; loads run STAGES - 1 steps ahead.
// Both kinds of LDS tile are XOR-swizzled in 16-byte chunks (by choosing the
// chunk that each lane fetches), so that fragment reads spread over the
// banks; a column operand's fragments come from transposing LDS reads.
//
// Everything outside an operand reads as zero: loads go through a buffer
// descriptor that ends with the operand's last valid byte of the step, and
// chunks past the end of the contraction are sent past the descriptor.  So no
// value in a gap or past an end, NaN or not, enters a sum, and rows and
// columns past the output are computed on repeated or zero values and never
// stored.
#pragma once

#include <mutex>
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
};

template <class ACC, int BM_, int BN_, int WGM_, int WGN_, bool A_COL, bool B_COL, int STAGES>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
    static constexpr int NW = WGM * WGN, THREADS = 64 * NW;
    static constexpr int WM = BM / WGM, WN = BN / WGN;
    static constexpr int FM = WM / 32, FN = WN / 32;
    static constexpr int KS = 4;                        // 32-byte slices of a step
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int LDS_BYTES = STAGES * STAGE;
    // Loads of 1 KB per stage and operand, issued by DW waves.  With 8 waves
    // only one wave of each SIMD (wave w runs on SIMD w % 4) loads, so the
    // other one only feeds the matrix pipe.
    static constexpr int DW = NW >= 8 ? NW / 2 : NW;
    static constexpr int AI = A_BYTES / 1024 / DW, BI = B_BYTES / 1024 / DW;
    static_assert(AI * DW * 1024 == A_BYTES && BI * DW * 1024 == B_BYTES, "whole loads per wave");
    static_assert(WM % 32 == 0 && WN % 32 == 0, "whole blocks per wave");
    static_assert(DW * 8 == 32, "the row swizzle alternates with the load");
    static_assert(!A_COL || BM >= 128, "column swizzle needs 16 chunks per row");
    static_assert(!B_COL || BN >= 128, "column swizzle needs 16 chunks per row");
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
    static constexpr int A_READS = A_COL ? 2 * FM : FM, B_READS = B_COL ? 2 * FN : FN;

    // Row tiles: 8 chunks of 16 bytes per row, chunk c of row m at c ^ swz.
    static __device__ __forceinline__ int row_swz(int m) { return (m ^ (m >> 3)) & 7; }
    // Column tiles: chunk c of contraction row k at c ^ swz.
    static __device__ __forceinline__ int col_swz(int k) { return 4 * (k & 3); }

    ACC acc[FM][FN];

    // Load i of an operand covers the rows from i * ROWS of its window: the
    // descriptor moves by ROWS rows and keeps the window's end, so rows past it
    // read as zero, and a lane's offset takes at most two values (the row
    // swizzle alternates with i).
    template <bool COL, int B> static constexpr int load_rows() {
        return COL ? DW * 64 / (B / 8) : DW * 8;
    }
    template <bool COL, int B>
    static __device__ __forceinline__ int load_chunk(int odd, int dwave, int lane) {
        if constexpr (COL) return (lane % (B / 8)) ^ col_swz(dwave * (64 / (B / 8)) + lane / (B / 8));
        else return (lane & 7) ^ row_swz(odd * 32 + dwave * 8 + lane / 8);
    }
    template <bool COL, int B>
    static __device__ __forceinline__ uint32_t load_offset(const Operand &o, int odd, int dwave, int lane) {
        const int row = COL ? dwave * (64 / (B / 8)) + lane / (B / 8) : dwave * 8 + lane / 8;
        return (uint32_t)row * (uint32_t)o.ld + (uint32_t)load_chunk<COL, B>(odd, dwave, lane) * 16u;
    }
    // Bytes of step kt's window, of which `left` (at most KE) elements, or
    // rows of a column operand, are valid; and its base.
    template <bool COL, int ELEM>
    static __device__ __forceinline__ uint32_t window_bytes(const Operand &o, int left) {
        if constexpr (COL) return (uint32_t)(left - 1) * (uint32_t)o.ld + (uint32_t)o.span;
        else return (uint32_t)(o.span - 1) * (uint32_t)o.ld + (uint32_t)(left * ELEM);
    }
    template <bool COL>
    static __device__ __forceinline__ const char *window_base(const Operand &o, int kt) {
        return o.base + (COL ? (int64_t)kt * 64 * o.ld : (int64_t)kt * 128);
    }
    template <int I, bool COL, int B>
    static __device__ __forceinline__ void load_part(const Operand &o, const char *base, uint32_t bytes,
                                                     uint32_t voff, uint32_t lds, int dwave) {
        const uint32_t skip = (uint32_t)I * load_rows<COL, B>() * (uint32_t)o.ld;
        load_to_lds(buffer_of(base + skip, bytes > skip ? bytes - skip : 0u), voff,
                    lds + (I * DW + dwave) * 1024);
    }
    template <bool COL, int B, int... I>
    static __device__ __forceinline__ void load_all(std::integer_sequence<int, I...>, const Operand &o,
                                                    const char *base, uint32_t bytes,
                                                    const uint32_t (&voff)[2], uint32_t lds, int dwave) {
        (load_part<I, COL, B>(o, base, bytes, voff[COL ? 0 : I & 1], lds, dwave), ...);
    }

    // Steps of a contraction of k elements, ELEM bytes each.
    template <int ELEM> static __device__ __forceinline__ int steps_of(int32_t k) {
        return (int)(((uint32_t)k + 128 / ELEM - 1) / (128 / ELEM));
    }

    // acc = A . B over a contraction of `k` elements (of a column operand:
    // rows; ELEM bytes each in a row operand).
    template <int ELEM>
    __device__ __forceinline__ void run(lds_t *smem, const Operand &a, const Operand &b, int32_t k) {
        constexpr int KE = 128 / ELEM;
        static_assert(!(A_COL || B_COL) || KE == 64, "column operands are bfloat16");
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WGN, wn = wave % WGN;
        const uint32_t smem_base = (uint32_t)(size_t)smem;
        const int KT = steps_of<ELEM>(k);
        const int dwave = wave < DW ? wave : 0;

        const uint32_t a_voff[2] = {load_offset<A_COL, BM>(a, 0, dwave, lane),
                                    A_COL ? 0u : load_offset<A_COL, BM>(a, 1, dwave, lane)};
        const uint32_t b_voff[2] = {load_offset<B_COL, BN>(b, 0, dwave, lane),
                                    B_COL ? 0u : load_offset<B_COL, BN>(b, 1, dwave, lane)};

        auto issue = [&](int kt, int st) __attribute__((always_inline)) {
            if (wave >= DW) return;                     // wave-uniform
            const int left = k - kt * KE < KE ? k - kt * KE : KE;
            uint32_t av[2] = {a_voff[0], a_voff[1]}, bv[2] = {b_voff[0], b_voff[1]};
            if (left < KE) {
                // the last step of a contraction that is no multiple of KE:
                // row chunks past its end are sent past the descriptor (a
                // column operand's rows past it lie there already)
                const int chunks = left * ELEM / 16;
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {
                    if (!A_COL && load_chunk<A_COL, BM>(odd, dwave, lane) >= chunks) av[odd] = 0xfffffff0u;
                    if (!B_COL && load_chunk<B_COL, BN>(odd, dwave, lane) >= chunks) bv[odd] = 0xfffffff0u;
                }
            }
            load_all<A_COL, BM>(std::make_integer_sequence<int, AI>{}, a, window_base<A_COL>(a, kt),
                                window_bytes<A_COL, ELEM>(a, left), av, smem_base + st * A_BYTES, dwave);
            load_all<B_COL, BN>(std::make_integer_sequence<int, BI>{}, b, window_base<B_COL>(b, kt),
                                window_bytes<B_COL, ELEM>(b, left), bv,
                                smem_base + STAGES * A_BYTES + st * B_BYTES, dwave);
        };

        // LDS addresses of this lane's fragments: few registers, and constants
        // for the reads' immediate field.  Row operand: 16 bytes of row
        // lane % 32; block i lies i * 4096 further, with the row swizzle of
        // i's parity.  Column operand: two transposing reads of 4 x 16 blocks,
        // of which this lane addresses row te, columns 4 tq..4 tq + 3; slices and
        // halves lie whole rows further, blocks differ in the swizzled chunk.
        constexpr int B_AT = STAGES * A_BYTES;
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
        auto load_frags = [&](int st, int ks, i32x4_t (&af)[FM], i32x4_t (&bf)[FN])
            __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if constexpr (A_COL) af[i] = col_read(a_at[0][i] + st * A_BYTES + ks * 16 * BM * 2, BM);
                else af[i] = *(lds_i32x4 *)(a_at[ks][i & 1] + st * A_BYTES + i * 4096);
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (B_COL) bf[j] = col_read(b_at[0][j] + st * B_BYTES + ks * 16 * BN * 2, BN);
                else bf[j] = *(lds_i32x4 *)(b_at[ks][j & 1] + st * B_BYTES + j * 4096);
            }
        };
        // Fragments are double-buffered in registers: the next slice's LDS
        // reads are spread between the current slice's matrix operations, and
        // a step's last slice is issued behind the next step's barrier, where
        // it covers the latency of that step's first reads.
        i32x4_t af[2][FM], bf[2][FN];
        auto mmas = [&](int fb) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mma(af[fb][i], bf[fb][j], acc[i][j]);
        };
        auto spread = [&]() __attribute__((always_inline)) {
            constexpr int R = A_READS + B_READS, M = FM * FN;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int n = (m + 1) * R / M - m * R / M;
                if (n == 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (n == 2) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                if (n == 3) __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
                if (n >= 4) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            }
        };
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s)
            if (s < KT) issue(s, s);
        auto step = [&](int kt, auto stage) __attribute__((always_inline)) {
            const int st = stage;
            // this wave's loads of step kt have landed (later steps' may be in
            // flight); behind the barrier every wave's have, and every wave
            // has read the stage that the next issue overwrites
            const int ahead = KT - 1 - kt;
            wait_groups<AI + BI, STAGES - 2>(ahead);
            lds_only_barrier();
            load_frags(st, 0, af[0], bf[0]);
            if (kt > 0) mmas(1);
            if (kt + STAGES - 1 < KT) {
                int to = st + STAGES - 1;
                if (to >= STAGES) to -= STAGES;
                issue(kt + STAGES - 1, to);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int ks = 0; ks + 1 < KS; ++ks) {
                load_frags(st, ks + 1, af[(ks + 1) & 1], bf[(ks + 1) & 1]);
                mmas(ks & 1);
                spread();
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if constexpr (STAGES == 2) {
            // two steps per turn: the stage is a constant, its offset goes
            // into the LDS reads' immediate field
            int kt = 0;
            for (; kt + 1 < KT; kt += 2) {
                step(kt, std::integral_constant<int, 0>{});
                step(kt + 1, std::integral_constant<int, 1>{});
            }
            if (kt < KT) step(kt, std::integral_constant<int, 0>{});
        } else {
            int st = 0;
            for (int kt = 0; kt < KT; ++kt) {
                step(kt, st);
                if (++st == STAGES) st = 0;
            }
        }
        if (KT > 0) mmas(1);
    }

    // Hands the tile out as f(row, column, v[RUN]) for runs of RUN columns (8,
    // or 1 where the output's rows are not aligned), each run once, whole rows
    // by neighbouring lanes.  Accumulators pass through LDS one 32-row block
    // row of every wave at a time: the direct layout would store 8 bytes per
    // row and instruction.  16-byte chunk c of a staged row r sits at
    // c ^ (r % 16).
    template <int RUN, class F>
    __device__ __forceinline__ void store(lds_t *smem, F f) const {
        static_assert(RUN == 8 || RUN == 1, "");
        constexpr int SROWS = WGM * 32, ROW = BN * 4, SBYTES = SROWS * ROW;
        constexpr bool TWICE = 2 * SBYTES <= LDS_BYTES;   // alternate between two halves
        static_assert(SBYTES <= LDS_BYTES, "a stripe fits");
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WGN, wn = wave % WGN;
        typedef __attribute__((address_space(3))) i32x4_t lds_i32x4;
        typedef __attribute__((address_space(3))) int32_t lds_i32;
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
            if constexpr (RUN == 8) {
                constexpr int LPR = BN / 8;
#pragma unroll
                for (int u = 0; u < SROWS * LPR; u += THREADS) {
                    const int rr = (u + tid) / LPR, c = (tid % LPR) * 2;
                    const i32x4_t lo = *(lds_i32x4 *)(s + rr * ROW + ((c ^ (rr & 15)) << 4));
                    const i32x4_t hi = *(lds_i32x4 *)(s + rr * ROW + (((c + 1) ^ (rr & 15)) << 4));
                    const int v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    f((rr >> 5) * WM + i * 32 + (rr & 31), (tid % LPR) * 8, v);
                }
            } else {
                for (int u = tid; u < SROWS * BN; u += THREADS) {
                    const int rr = u / BN, c = u % BN;
                    const int v[1] = {*(lds_i32 *)(s + rr * ROW + (((c >> 2) ^ (rr & 15)) << 4) + (c & 3) * 4)};
                    f((rr >> 5) * WM + i * 32 + (rr & 31), c, v);
                }
            }
        }
    }
};

// Launches a kernel with dynamic LDS, whose limit is a per-device attribute of
// the kernel: set once per device (thread-safe).
template <auto KERNEL, class ARGS>
inline hipError_t launch_lds(int64_t blocks, int threads, int lds_bytes, hipStream_t s, const ARGS &a) {
    constexpr int kMaxDevices = 64;
    static std::once_flag once[kMaxDevices];
    static hipError_t set[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
        return hipErrorInvalidDevice;
    std::call_once(once[dev], [dev, lds_bytes] {
        set[dev] = hipFuncSetAttribute((const void *)KERNEL,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, lds_bytes);
    });
    if (set[dev] != hipSuccess) return set[dev];
    hipLaunchKernelGGL(KERNEL, dim3((unsigned)blocks), dim3(threads), lds_bytes, s, a);
    return hipGetLastError();
}

}  // namespace ffn
}  // namespace gemm_rs
