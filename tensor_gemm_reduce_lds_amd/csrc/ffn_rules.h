// Which kernel a call of the 8-bit product, the row quantisation or the products
// grouped by expert takes: rules on sizes from measured times.  Plain C++, so that
// a host check can ask which kernel a size reaches.
#pragma once

#include <math.h>
#include <stdint.h>

namespace gemm_rs {
namespace ffn {

constexpr int kCus = 256;   // MI355X: 8 XCDs x 32 CUs

inline double ceil_div(double a, double b) { return ceil(a / b); }

// ---- 8-bit product ---------------------------------------------------------
enum Q8Choice {
    kQ8Rows16, kQ8Rows16Wide, kQ8Rows32, kQ8Rows32Wide, kQ8Rows64, kQ8Rows64Wide,
    kQ8Tile256, kQ8Tile128, kQ8Tile128Deep, kQ8Tile64x128, kQ8Tile64x128Deep, kQ8Tile64,
    kQ8Choices
};

inline Q8Choice q8_choice(int64_t M, int64_t N) {
    // Up to 64 rows the product is bound by streaming w: as many workgroups as
    // there are CUs, so 32 channels each (wide) where that still makes 256 of
    // them (the rows of a are then read half as often), else 16.  Measured, us for
    // 16 / 32 channels: 64 x 8192 x 3584 11.7 / 9.7, 64 x 3584 x 8192 10.5 / 14.1.
    // From 65 rows on the tiles are as fast or faster (128 rows in such streams
    // against 64 x 64 tiles: 128 x 8192 x 3584 14.6 / 11.5, 128 x 3584 x 8192
    // 17.8 / 18.6, 71 x 5241 x 6656 26.4 / 17.6; 64 rows: 64 x 3584 x 8192 10.4 /
    // 18.2).
    const bool wide = N >= 32 * kCus;
    if (M <= 16) return wide ? kQ8Rows16Wide : kQ8Rows16;
    if (M <= 32) return wide ? kQ8Rows32Wide : kQ8Rows32;
    if (M <= 64) return wide ? kQ8Rows64Wide : kQ8Rows64;
    // The tile with the least time, from the rounds of 256 workgroups that it
    // makes (a round costs about as much where it is not full) and times
    // measured at K = 3584, in us.  Large tiles read fewer bytes per operation,
    // small ones fill the CUs when there are few.  One round takes deep loads
    // and one workgroup per CU, more rounds two or three per CU.  Measured, us
    // for 256 x 256, 128 x 128 (deep / two per CU), 64 x 128 (deep / three), 64 x
    // 64: 8192 x 8192 x 3584 236, 354 / 306, 359 / -, 422; 1024 x 3584 x 8192 78,
    // 39 / 44, 44 / 46, 57; 512 x 3584 x 8192 78, 31 / 38, 27 / 39, 28; 256 x 3584
    // x 8192 76, 30 / -, 24 / -, 19; 1000 x 4104 x 1792 -, 24 / 21, - / 18, 21.
    // (K does not enter: a tile's fixed part, its first loads and last stores,
    // weighs more in a short contraction than these times have it.)
    auto rounds = [&](int64_t bm, int64_t bn) {
        return (double)((((M + bm - 1) / bm) * ((N + bn - 1) / bn) + kCus - 1) / kCus);
    };
    const double r128 = rounds(128, 128), r64w = rounds(64, 128);
    const double t256 = 59 * rounds(256, 256), t128 = r128 <= 1 ? 18 : 20 * r128;
    const double t64w = r64w <= 1 ? 13 : 4 + 11 * r64w, t64 = 2 + 8 * rounds(64, 64);
    if (t256 <= t128 && t256 <= t64w && t256 <= t64) return kQ8Tile256;
    if (t128 <= t64w && t128 <= t64) return r128 <= 1 ? kQ8Tile128Deep : kQ8Tile128;
    if (t64w <= t64) return r64w <= 1 ? kQ8Tile64x128Deep : kQ8Tile64x128;
    return kQ8Tile64;
}

// ---- row quantisation -------------------------------------------------------
// A wave per row where there are many short rows, else a workgroup; rows of more
// than 16384 columns are read twice instead of held.
enum QuantChoice { kQuantWave, kQuant2048, kQuant8192, kQuant16384, kQuantTwice, kQuantChoices };

inline QuantChoice quant_choice(int64_t rows, int64_t cols) {
    if (cols <= 2048) return rows >= kCus ? kQuantWave : kQuant2048;
    return cols <= 8192 ? kQuant8192 : cols <= 16384 ? kQuant16384 : kQuantTwice;
}

// ---- products grouped by expert, NN and NT ------------------------------------
enum RowsChoice { kRows256, kRows128x256, kRows128, kRows128Deep, kRows64x128, kRowsStream, kRowsChoices };

// The tile with the least time, which is taken as rounds of 256 workgroups (a round
// costs about as much where it is not full) times the steps of 64 times `step`,
// plus `fixed` (the first loads, the last stores, waiting for the memory that all
// of them want at once), in us, but not less than the operands take at 5 TB/s, a
// copy's rate.  Row tiles are counted as far as the host can tell: every expert
// with rows has one that is half empty; what other splits cost over even ones
// (16384 rows, 8 experts of 4096 x 3584, one with half of the rows 416 us, with all
// 391, even 406; 8000 rows, 64 experts of 4096 x 1792, one with half 220, 8 with
// three quarters 232, even 188) is their row tiles.  step and fixed are fitted to
// the times of 170 calls of 1..16384 rows, sizes 256..4096, 1..64 experts, where
// the choice is 1% slower than the best on average.  These and the following are
// times of calls repeated on the same operands, part of which the caches hold.
// Large tiles do the most work per byte, small ones fill the CUs; of equals the
// larger, which reads B less often where an expert has more rows than the mean.
// Measured, us for 256 x 256, 128 x 256, 128 x 128 (deep loads, one workgroup per
// CU / two per CU), 64 x 128, 32 x 64 streams (rows : K : N : E): 16384 : 4096 :
// 3584 : 8 435, 500, 576 / 509, 679, 1420; 8000 : 4096 : 1792 : 64 235, 224, 245 /
// 237, 266, 463; 10807 : 896 : 1408 : 1 51, 40, 46 / 37, 46, 144; 512 : 4096 : 3584
// : 8 75, 69, 50 / 53, 74, 88; 1160 : 1088 : 960 : 6 26, 18, 12 / 13, 10, 18; 128 :
// 2048 : 1024 : 1 26, 27, 17 / 18, 13, 8.4.
inline RowsChoice rows_choice(int64_t rows, int64_t K, int64_t N, int64_t E) {
    struct Option {
        int bm, bn;
        double step, fixed;
    };
    const Option options[] = {{256, 256, 1.76, 15.6}, {128, 256, 1.13, 8.0}, {128, 128, 0.71, 1.3},
                              {64, 128, 0.47, 1.4}, {32, 64, 0.22, 1.4}};
    const double live = (double)(E < rows ? E : rows), steps = ceil_div((double)K, 64);
    const double floor_us = 2.0 * (live * K * N + (double)rows * (K + N)) / 5.0e6;
    int best = 0;
    double best_us = 0, best_rounds = 0;
    for (int i = 0; i < 5; ++i) {
        const Option &o = options[i];
        double row_tiles = (double)rows / o.bm + live / 2;
        if (row_tiles < live) row_tiles = live;
        const double rounds = ceil_div(row_tiles * ceil_div((double)N, o.bn), kCus);
        double us = rounds * (steps * o.step + o.fixed);
        if (us < floor_us) us = floor_us;
        if (i == 0 || us < 0.97 * best_us) {
            best = i;
            best_us = us;
            best_rounds = rounds;
        }
    }
    switch (best) {
    case 0: return kRows256;
    case 1: return kRows128x256;
    case 2: return best_rounds > 1 ? kRows128 : kRows128Deep;
    case 3: return kRows64x128;
    default: return kRowsStream;
    }
}

// ---- products grouped by expert, TN -------------------------------------------
// 256 x 256 tiles, which read the rows half as often, or 128 x 128 with two
// workgroups per CU, so that one stores while the other loads.  With four rounds of
// large tiles or more these are as fast where the caches hold the rows and faster
// where they do not, as behind other work (us after a pass over 1 GB, for 256 /
// 128: 6001 rows, 32 experts of 2048 x 1792 in 32 bits 136 / 165, 8000 rows, 64
// experts of 4096 x 1792 in bfloat16 321 / 404, 16384 rows, 8 experts of 4096 x
// 3584 427 / 570).  With one to four rounds they mostly are where groups are long,
// as the last round counts less (the same in bfloat16, 8 experts of 2048 x 2048, 512
// tiles: 448 rows each 45 / 58, 1024 77 / 99; of 1536 x 1536, 288 tiles: 448 rows
// 40 / 39, 1024 70 / 65, 4096 222 / 213, but repeated on the same rows 168 / 196);
// with shorter groups it depends (221 rows each, 9 experts of 1920 x 1840: 48 / 44,
// repeated 35 / 31; 256 rows each, 8 experts of 2048 x 2048: 36 / 47, repeated 28 /
// 31).  With few of the small ones too, `parts` workgroups share a tile's rows and
// a second kernel adds them, as many as take the least time, from about 0.5 us per
// step of 64 rows, and for the second kernel 4 us and the parts' traffic (16030
// rows, 1296 x 304, 2 experts: 1 part 76 us, 4 38, 8 32; 7984 rows, 768 x 512, 8
// experts: 1 part 20 us, 2 26).
struct TnChoice {
    bool large;
    int parts;
};
inline TnChoice tn_choice(int64_t rows, int64_t K, int64_t N, int64_t E) {
    const int64_t large = E * ((K + 255) / 256) * ((N + 255) / 256);
    const int64_t small = E * ((K + 127) / 128) * ((N + 127) / 128);
    if (large >= 4 * kCus || (large >= kCus && rows / E >= 448)) return {true, 1};
    const double steps = (double)(rows / E) / 64, part_us = (double)E * K * N * 8 / 6.0e6;
    int parts = 1;
    double best_us = 0.5 * steps;
    for (int p = 2; p <= 16 && p * small <= 2 * kCus; ++p) {
        const double us = 0.5 * steps / p + 4 + p * part_us;
        if (us < best_us) {
            parts = p;
            best_us = us;
        }
    }
    return {false, parts};
}

}  // namespace ffn
}  // namespace gemm_rs
