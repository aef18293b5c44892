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
    for (int i = 0; i < kTiles; ++i) {
        const gbx::TileCost &t = kRowTiles[i];
        const double tiles = gbx::row_tiles(T, E, t.bm) * ceil((double)cols / t.bn);
        // The slices of 64 rows of a multiple of 2 KiB lie in few memory channels: 1.1 to 1.3 times as long (1 x 14336 x 4096
        // 17.6 us, the streaming kernel 14.6; 1 x 11016 x 512 no longer).
        const double few = t.bm <= 64 && K % 2048 == 0 ? 1.3 : 1.0;
        for (int s : gbx::kSplits) {
            if (s > 1 && (2 * s > slices || (double)s * T * cols * 4.0 > (double)workspace)) break;
            consider(few * (gbx::ring_cost(t, tiles * s, ceil(slices / s), cus) + (s > 1 ? kSecondPass + 2.0 * s * T * cols * 4.0 / 4.0e6 : 0)),
                     {GBM_RING, i, s});
        }
    }
    // The persistent kernel's stream needs two slices.
    const double tiles = gbx::row_tiles(T, E, 256) * ceil(cols / 256.0);
    if (slices >= 2)
        consider(ceil(tiles / cus) * (kBig.fix + slices * (2 * tiles > cus ? kBig.slice : kBig.latency)), {GBM_PERSISTENT, 0, 1});
    // Few rows an expert: each workgroup reads them again.
    if (T <= 8 * some) {
        const double n = gbx::row_tiles(T, E, 16) * ceil(cols / 16.0) / cus;
        consider(1.2 + fmax(n * (kStream.fix + slices * kStream.slice), 2 + slices * kStream.latency), {GBM_STREAM, 0, 1});
    }
    return best;
}

}  // namespace gbm
