// Choice of kernel, tile and K split for an 8-bit product (host only).
#pragma once

#include "../experts/gx_plan.hpp"
#include "gba_moe.h"
#include "gm_launch.hpp"

namespace gbm {

struct Plan {
    int kind;     // GBM_RING, ...
    int tile;     // ring kernel: its tile
    int splits;
};

// What a tile costs in microseconds, as gx_plan.hpp's (a slice is 128 values). Measured on one MI355X over 190 drawn
// sizes (1 to 16384 rows, 1 to 64 experts, 512 to 14336 columns, depths of 512 to 14336), every tile and splits of 1, 2 and
// 4 of each, with weights that the caches do not hold: with these the choice was 2.8 % slower than the best on
// average, 33 % at most (4863 rows of 16 experts: their uneven shares are not known here).
constexpr gbx::TileCost kRowTiles[kTiles] = {{16, 64, 1.5, 0.225, 0.14}, {32, 64, 0.93, 0.21, 0.185}, {64, 64, 0.95, 0.26, 0.25},
                                             {64, 128, 1.65, 0.45, 0.30}, {128, 64, 1.1, 0.435, 0.44}, {128, 128, 2.3, 0.60, 0.75}};
constexpr gbx::TileCost kBig = {256, 256, 9.0, 1.3, 1.14};
constexpr gbx::TileCost kStream = {16, 16, 0.1, 0.08, 0.075};   // tiles a CU share its memory: no rounds
// Staged or streamed, measured over 2350 sizes (1 to 8 rows on each of 1 to 64 experts, 72 to 28672 columns, depths of 256 to
// 14464, weights that no cache holds): with these 1.6 % slower than the better one on average, 63 % at most (256 rows on 64
// experts of 14336 x 256, 126 us streamed and 77 staged). Both take as long as HBM takes for the weights at least, which the
// staged kernel's own cost does not show, the streaming one 5 % more for each further row.
constexpr double kStaged = 1.05, kStagedStart = 2, kStagedRate = 6.3e6, kStreamRate = 6.2e6, kRowRead = 0.05;   // us, bytes / us
// A depth of a multiple of 2 KiB, whose rows lie in fewer memory channels, costs tiles of up to 64 rows little: 1 x 4096 x 3968
// 10.7 us, x 4096 11.1, x 4224 12.2; 1 x 14336 13.6, 15.2, 14.4; 96 x 14336 18.1, 19.7, 19.2. Below this many columns such tiles
// count 1.3 times all the same, and plans stay what they have been; that is no gain either: of 355 sizes of 40 to 400
// columns it takes 15 % longer on average (4111 rows of 13 experts, 264 x 4096, 31.4 us and 21.7 without; 8000 rows of 70, 264 x
// 14336, 106 and 126).
constexpr int kNarrow = 512;
constexpr double kSecondPass = 2.3;                             // a launch behind another one

inline Plan plan_f8(int64_t T, int64_t E, int64_t cols, int64_t K, size_t workspace, int cus) {
    const double slices = ceil(K / 128.0), some = E < T ? E : T;
    Plan best = {GBM_RING, gbx::TILE_16x64, 1};
    double least = 1e300;
    auto consider = [&](double cost, const Plan &p) {
        if (cost < least) {
            least = cost;
            best = p;
        }
    };
    // Narrow outputs, rows of a multiple of 2 KiB: see kNarrow.
    const double few = cols < kNarrow && K % 2048 == 0 ? 1.3 : 1.0;
    double ring = 0;
    for (int i = 0; i < kTiles; ++i) {
        const gbx::TileCost &t = kRowTiles[i];
        const double tiles = gbx::row_tiles(T, E, t.bm) * ceil((double)cols / t.bn);
        for (int s : gbx::kSplits) {
            if (s > 1 && (2 * s > slices || (double)s * T * cols * 4.0 > (double)workspace)) break;
            const double cost = gbx::ring_cost(t, tiles * s, ceil(slices / s), cus) + (s > 1 ? kSecondPass + 2.0 * s * T * cols * 4.0 / 4.0e6 : 0);
            if ((t.bm <= 64 ? few : 1.0) * cost < least) ring = cost;
            consider((t.bm <= 64 ? few : 1.0) * cost, {GBM_RING, i, s});
        }
    }
    least = ring;
    // The persistent kernel's stream needs two slices.
    const double tiles = gbx::row_tiles(T, E, 256) * ceil(cols / 256.0);
    if (slices >= 2)
        consider(ceil(tiles / cus) * (kBig.fix + slices * (2 * tiles > cus ? kBig.slice : kBig.latency)), {GBM_PERSISTENT, 0, 1});
    // Few rows an expert: each workgroup reads them again.
    if (T <= 8 * some) {
        const double n = gbx::row_tiles(T, E, 16) * ceil(cols / 16.0) / cus, read = some * cols * K;
        const double cost = fmax(1.2 + fmax(n * (kStream.fix + slices * kStream.slice), 2 + slices * kStream.latency),
                                 read / kStreamRate * (1 + kRowRead * (T / some - 1)));
        if (cost < fmax(kStaged * least, kStagedStart + read / kStagedRate)) best = {GBM_STREAM, 0, 1};
    }
    return best;
}

}  // namespace gbm
