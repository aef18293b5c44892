// Choice of kernel, tile and K split for a grouped product (host only).
#pragma once

#include <math.h>

#include "gx_launch.hpp"

namespace gbx {

// What a tile costs in microseconds: `fix` (start and epilogue) and `slice` (one
// 64-word K slice) where its CU is full, and the slice's latency where a
// workgroup has its CU to itself. Measured on one MI355X over 1 to 1000 rows an
// expert, 1 to 32 experts, 1024 to 14336 columns and depths of 1024 to 4096, in
// 16 and in 4 bits (a 64-word slice is 64 or 256 values deep): with these the
// choice was 2.2 % slower than the best on average, 37 % at most (a gradient of 18 us).
struct TileCost {
    int bm, bn;
    double fix, slice, latency;
};
constexpr TileCost kRowTiles[kTiles] = {{16, 64, 1.15, 0.18, 0.17}, {32, 64, 1.65, 0.18, 0.24},
                                        {64, 64, 1.5, 0.26, 0.34},  {64, 128, 2.4, 0.35, 0.48},
                                        {128, 64, 1.9, 0.43, 0.53}, {128, 128, 2.9, 0.65, 0.72}};
constexpr TileCost kGradTileCost[kGradTiles] = {{64, 64, 1.65, 0.27, 0.36}, {128, 128, 2.55, 0.68, 0.79}};
constexpr TileCost kBig = {256, 256, 7.0, 1.6, 1.25};

struct Plan {
    bool big;       // persistent 256 x 256 kernel
    int tile;       // ring kernel's tile otherwise
    int splits;
    bool stream;    // B is read non-temporally
};

inline double ring_cost(const TileCost &t, double tiles, double slices, double cus) {
    const double n = tiles / cus, full = n < 3 ? fmax(1, ceil(n - 0.1)) : n;   // tiles a CU runs
    const double alone = t.fix + 2 + slices * t.latency, shared = full * (t.fix + slices * t.slice);
    return alone > shared ? alone : shared;
}

// The persistent kernel runs whole rounds of one tile a CU; with half of the CUs
// or fewer at work a slice takes less.
inline double big_cost(double tiles, double slices, double cus) {
    return ceil(tiles / cus) * (kBig.fix + slices * (2 * tiles > cus ? kBig.slice : kBig.latency));
}

// Adds the second pass: a launch, and the partial sums written and read at 4 TB/s.
inline double reduce_cost(double values, int splits) { return 5.0 + 2.0 * splits * values * 4.0 / 4.0e6; }

constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};

// Row tiles that T rows of E experts make, as far as the host can tell: half a
// tile more for each expert with rows; exact for one expert.
inline double row_tiles(double T, double E, int bm) {
    if (E == 1) return ceil(T / bm);
    const double some = E < T ? E : T, guess = T / bm + 0.5 * some;
    return guess > some ? guess : some;
}

// Rows mode: T rows, `cols` columns, a depth of `words` 16-bit words.
inline Plan plan_rows(int64_t T, int64_t E, int64_t cols, int64_t words, size_t workspace, int cus) {
    const double slices = ceil(words / 64.0);
    Plan best = {false, TILE_16x64, 1, false};
    double least = 1e300;
    for (int i = 0; i < kTiles; ++i) {
        const TileCost &t = kRowTiles[i];
        const double tiles = row_tiles(T, E, t.bm) * ceil((double)cols / t.bn);
        for (int s : kSplits) {
            if (s > 1 && (2 * s > slices || (double)s * T * cols * 4.0 > (double)workspace)) break;
            const double c = ring_cost(t, tiles * s, ceil(slices / s), cus) + (s > 1 ? reduce_cost((double)T * cols, s) : 0);
            if (c < least) {
                least = c;
                best = {false, i, s, false};
            }
        }
    }
    // The persistent kernel's stream needs two slices.
    if (slices >= 2 && big_cost(row_tiles(T, E, 256) * ceil(cols / 256.0), slices, cus) < least) best = {true, 0, 1, false};
    // B read once (about one row tile an expert), and what one call reads of it, at most min(E, T)
    // experts, too large for the 256 MiB cache behind the L2 to hold until the next
    // call: read non-temporally (12 of 32 experts of 2816 x 2048 bf16, 16 rows: 36 -> 32 us; a B that
    // the cache holds is 10 to 25 % slower so). Up to five such tiles a CU are then split in four where that
    // gains more than the second pass takes. Two things are lost whole: the CUs' last round of
    // tiles is half empty on average, 0.08 us a slice; and rows of a multiple of 4 KiB lie in
    // few memory channels, which four places along K spread out, 0.08 us a slice and tile a CU up to
    // two. Measured for 1 to 4 rows on 8 experts, over 0.5 to 5 tiles a CU, split against whole: rows of
    // 30 slices +9 % (-5 to +26), 40 +3 % (-8 to +19); of 32 slices, 4 KiB, -4 % (-14 to +7), 64 -9 %
    // (-22 to -2). 12 of 32 experts of 2816 x 2048: 34 -> 28 us.
    const double some = E < T ? E : T, b_bytes = 2.0 * some * cols * words;
    const TileCost &t = kRowTiles[best.tile];
    if (!best.big && t.bm <= 64 && T / some <= t.bm && b_bytes > 128.0 * 1024 * 1024) {
        best.stream = true;
        const double n = row_tiles(T, E, t.bm) * ceil((double)cols / t.bn) / cus;
        const double lost = slices * (0.08 + (words % 2048 == 0 ? 0.08 * fmin(n, 2) : 0));
        if (t.bm <= 32 && best.splits == 1 && n <= 5 && lost > reduce_cost((double)T * cols, 4) &&
            16.0 * T * cols <= (double)workspace)
            best.splits = 4;
    }
    return best;
}

// Weight gradients: E products of M x N, summed over T / E rows on average. With
// the bias gradient (`sums`) the ring kernel costs another launch, the persistent one does
// not. (The column sums of few long experts take longer than a launch, one of 16384 rows 29 us;
// the persistent kernel has few tiles there and is no choice: with the measured time in place of 4 us
// no plan of one to four experts from 2048 rows on changes.)
inline Plan plan_grad(int64_t T, int64_t E, int64_t M, int64_t N, bool sums, size_t workspace, int cus) {
    const double slices = ceil((double)T / E / 64.0);
    Plan best = {false, GRAD_64x64, 1, false};
    double least = 1e300;
    for (int i = 0; i < kGradTiles; ++i) {
        const TileCost &t = kGradTileCost[i];
        const double tiles = (double)E * ceil((double)M / t.bm) * ceil((double)N / t.bn);
        for (int s : kSplits) {
            if (s > 1 && (2 * s > slices || (double)s * E * M * N * 4.0 > (double)workspace)) break;
            const double c = ring_cost(t, tiles * s, ceil(slices / s), cus) + (s > 1 ? reduce_cost((double)E * M * N, s) : 0) +
                             (sums ? 4.0 : 0.0);
            if (c < least) {
                least = c;
                best = {false, i, s, false};
            }
        }
    }
    const double tiles = (double)E * ceil(M / 256.0) * ceil(N / 256.0);
    if (big_cost(tiles, slices < 2 ? 2 : slices, cus) < least) best = {true, 0, 1, false};
    return best;
}

}  // namespace gbx
