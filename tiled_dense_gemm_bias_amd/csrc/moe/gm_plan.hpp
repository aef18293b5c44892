// Choice of tile and K split for an 8-bit product (host only).
#pragma once

#include "../experts/gx_plan.hpp"

namespace gbm {

using gbx::Plan;

constexpr gbx::TileCost kBig = {256, 256, 8.0, 1.75, 1.4};

inline Plan plan_f8(int64_t T, int64_t E, int64_t cols, int64_t K, size_t workspace, int cus) {
    const double slices = ceil(K / 128.0);
    Plan best = {false, gbx::TILE_16x64, 1, false};
    double least = 1e300;
    for (int i = 0; i < gbx::kTiles; ++i) {
        const gbx::TileCost &t = gbx::kRowTiles[i];
        const double tiles = gbx::row_tiles(T, E, t.bm) * ceil((double)cols / t.bn);
        for (int s : gbx::kSplits) {
            if (s > 1 && (2 * s > slices || (double)s * T * cols * 4.0 > (double)workspace)) break;
            const double c = gbx::ring_cost(t, tiles * s, ceil(slices / s), cus) + (s > 1 ? gbx::reduce_cost((double)T * cols, s) : 0);
            if (c < least) {
                least = c;
                best = {false, i, s, false};
            }
        }
    }
    // The persistent kernel's stream needs two slices.
    const double tiles = gbx::row_tiles(T, E, 256) * ceil(cols / 256.0);
    if (slices >= 2 && ceil(tiles / cus) * (kBig.fix + slices * (2 * tiles > cus ? kBig.slice : kBig.latency)) < least) best = {true, 0, 1, false};
    return best;
}

}  // namespace gbm
