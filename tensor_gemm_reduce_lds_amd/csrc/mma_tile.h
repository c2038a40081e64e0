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
    static_assert(!A_COL || BM >= 128, "column swizzle needs 16 chunks per row");
    static_assert(!B_COL || BN >= 128, "column swizzle needs 16 chunks per row");
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
    static constexpr int A_READS = A_COL ? 2 * FM : FM, B_READS = B_COL ? 2 * FN : FN;

    // Row tiles: 8 chunks of 16 bytes per row, chunk c of row m at c ^ swz.
    static __device__ __forceinline__ int row_swz(int m) { return (m ^ (m >> 3)) & 7; }
    // Column tiles: chunk c of contraction row k at c ^ swz.
    static __device__ __forceinline__ int col_swz(int k) { return 4 * (k & 3); }

    ACC acc[FM][FN];

    // Byte offset (inside a step's window) that this lane loads in issue i.
    template <bool COL, int B>
    static __device__ __forceinline__ uint32_t load_offset(const Operand &o, int i, int dwave, int lane) {
        if constexpr (COL) {
            constexpr int CPR = B / 8;                  // chunks per contraction row
            const int k = (i * DW + dwave) * (64 / CPR) + lane / CPR;
            return (uint32_t)(k * o.ld + ((lane % CPR) ^ col_swz(k)) * 16);
        } else {
            int m = (i * DW + dwave) * 8 + lane / 8;
            const int c = (lane & 7) ^ row_swz(m);
            if (m >= o.span) m = o.span - 1;            // rows past the end repeat the last
            return (uint32_t)(m * o.ld + c * 16);
        }
    }
    // Descriptor of step kt, of which `left` (at most KE) elements, or rows of
    // a column operand, are valid.
    template <bool COL, int ELEM>
    static __device__ __forceinline__ i32x4_t window(const Operand &o, int kt, int left) {
        if constexpr (COL)
            return buffer_of(o.base + (int64_t)kt * 64 * o.ld, (uint32_t)(left - 1) * (uint32_t)o.ld + (uint32_t)o.span);
        else
            return buffer_of(o.base + (int64_t)kt * 128,
                             (uint32_t)(o.span - 1) * (uint32_t)o.ld + (uint32_t)(left * ELEM));
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
        const int KT = (int)(((uint32_t)k + KE - 1) / KE);
        const int dwave = wave < DW ? wave : 0;

        uint32_t a_voff[AI], b_voff[BI];
#pragma unroll
        for (int i = 0; i < AI; ++i) a_voff[i] = load_offset<A_COL, BM>(a, i, dwave, lane);
#pragma unroll
        for (int i = 0; i < BI; ++i) b_voff[i] = load_offset<B_COL, BN>(b, i, dwave, lane);

        auto issue = [&](int kt, int st) __attribute__((always_inline)) {
            if (wave >= DW) return;                     // wave-uniform
            const int left = k - kt * KE < KE ? k - kt * KE : KE;
            const uint32_t As = smem_base + st * A_BYTES;
            const uint32_t Bs = smem_base + STAGES * A_BYTES + st * B_BYTES;
            const i32x4_t ra = window<A_COL, ELEM>(a, kt, left), rb = window<B_COL, ELEM>(b, kt, left);
            if (left == KE) {
#pragma unroll
                for (int i = 0; i < AI; ++i) load_to_lds(ra, a_voff[i], As + (i * DW + dwave) * 1024);
#pragma unroll
                for (int i = 0; i < BI; ++i) load_to_lds(rb, b_voff[i], Bs + (i * DW + dwave) * 1024);
            } else {
                // the last step of a contraction that is no multiple of KE:
                // row chunks past its end are sent past the descriptor (a
                // column operand's rows past it lie there already)
                const int chunks = left * ELEM / 16;
                auto cut = [&](uint32_t voff, int i) __attribute__((always_inline)) {
                    const int m = (i * DW + dwave) * 8 + lane / 8;
                    return ((lane & 7) ^ row_swz(m)) < chunks ? voff : 0xfffffff0u;
                };
#pragma unroll
                for (int i = 0; i < AI; ++i)
                    load_to_lds(ra, A_COL ? a_voff[i] : cut(a_voff[i], i), As + (i * DW + dwave) * 1024);
#pragma unroll
                for (int i = 0; i < BI; ++i)
                    load_to_lds(rb, B_COL ? b_voff[i] : cut(b_voff[i], i), Bs + (i * DW + dwave) * 1024);
            }
        };

        // LDS offsets of this lane's fragments inside a stage's tile.  Row
        // operand: 16 bytes of row lane % 32.  Column operand: two
        // transposing reads of 4 x 16 blocks, of which this lane addresses
        // row e, columns 4q..4q+3.
        int a_off[FM][KS][A_COL ? 2 : 1], b_off[FN][KS][B_COL ? 2 : 1];
        const int grp = lane >> 4, te = (lane & 15) >> 2, tq = lane & 3;
        auto col_off = [&](int x, int ks, int h, int width) __attribute__((always_inline)) {
            const int kk = ks * 16 + 8 * (grp >> 1) + 4 * h + te;
            const int n = x + 16 * (grp & 1) + 4 * tq;
            return kk * (width * 2) + (((n >> 3) ^ col_swz(kk)) << 4) + ((n & 7) << 1);
        };
        auto row_off = [&](int x, int ks) __attribute__((always_inline)) {
            const int m = x + (lane & 31), c = 2 * ks + (lane >> 5);
            return m * 128 + ((c ^ row_swz(m)) << 4);
        };
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if constexpr (A_COL) {
                    a_off[i][ks][0] = col_off(wm * WM + i * 32, ks, 0, BM);
                    a_off[i][ks][1] = col_off(wm * WM + i * 32, ks, 1, BM);
                } else {
                    a_off[i][ks][0] = row_off(wm * WM + i * 32, ks);
                }
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (B_COL) {
                    b_off[j][ks][0] = STAGES * A_BYTES + col_off(wn * WN + j * 32, ks, 0, BN);
                    b_off[j][ks][1] = STAGES * A_BYTES + col_off(wn * WN + j * 32, ks, 1, BN);
                } else {
                    b_off[j][ks][0] = STAGES * A_BYTES + row_off(wn * WN + j * 32, ks);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = ACC{};

        auto col_read = [&](lds_t *at, const int (&off)[2]) __attribute__((always_inline)) {
            typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
            const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(at + off[0]));
            const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(at + off[1]));
            const i16x8_t both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(i32x4_t, both);
        };
        auto load_frags = [&](int st, int ks, i32x4_t (&af)[FM], i32x4_t (&bf)[FN])
            __attribute__((always_inline)) {
            lds_t *const SA = smem + st * A_BYTES, *const SB = smem + st * B_BYTES;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if constexpr (A_COL) af[i] = col_read(SA, a_off[i][ks]);
                else af[i] = *(__attribute__((address_space(3))) i32x4_t *)(SA + a_off[i][ks][0]);
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (B_COL) bf[j] = col_read(SB, b_off[j][ks]);
                else bf[j] = *(__attribute__((address_space(3))) i32x4_t *)(SB + b_off[j][ks][0]);
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

    // Hands the tile out as f(row, column, v[8]) for runs of 8 columns, each
    // run once, whole rows by neighbouring lanes.  Accumulators pass through
    // LDS one 32-row block row of every wave at a time: the direct layout
    // would store 8 bytes per row and instruction.  16-byte chunk c of a
    // staged row r sits at c ^ (r % 16).
    template <class F>
    __device__ __forceinline__ void store(lds_t *smem, F f) const {
        constexpr int SROWS = WGM * 32, ROW = BN * 4, SBYTES = SROWS * ROW;
        constexpr int LPR = BN / 8, RPI = 64 / LPR;
        constexpr bool TWICE = 2 * SBYTES <= LDS_BYTES;   // alternate between two halves
        static_assert(SBYTES <= LDS_BYTES, "a stripe fits");
        constexpr int PER_WAVE = SROWS / NW;
        static_assert(PER_WAVE % RPI == 0, "whole rows per wave");
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wave / WGN, wn = wave % WGN;
        typedef __attribute__((address_space(3))) i32x4_t lds_i32x4;
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
#pragma unroll
            for (int r = 0; r < PER_WAVE; r += RPI) {
                const int rr = wave * PER_WAVE + r + lane / LPR, c = (lane % LPR) * 2;
                const i32x4_t lo = *(lds_i32x4 *)(s + rr * ROW + ((c ^ (rr & 15)) << 4));
                const i32x4_t hi = *(lds_i32x4 *)(s + rr * ROW + (((c + 1) ^ (rr & 15)) << 4));
                const int v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                f((rr >> 5) * WM + i * 32 + (rr & 31), (lane % LPR) * 8, v);
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
