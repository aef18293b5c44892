// Tables of the products' kernel instances, one translation unit each (the device pass instantiates
// the kernels, the host pass defines the table). Tiles as gx_launch.hpp's.
#pragma once

#include "../experts/gx_launch.hpp"

namespace gbm {

using gbx::Group;
using gbx::kTiles;
using gbx::LaunchFn;

extern const LaunchFn f8_act[2][kTiles], f8_slope[2][kTiles];   // [output type][tile]
extern const LaunchFn f8_part[kTiles];

}  // namespace gbm

#define GBM_KERNEL_(BM, BN, WM, WN, ST, DT, EPI) \
    template __global__ void gbx::grouped_ring_kernel<BM, BN, WM, WN, ST, gbx::OP_F8, DT, gbx::EPI, true, false>(gbx::Group);
#define GBM_LAUNCH_(BM, BN, WM, WN, ST, DT, EPI) gbx::launch_ring<BM, BN, WM, WN, ST, gbx::OP_F8, DT, gbx::EPI, true, false>,
#ifdef __HIP_DEVICE_COMPILE__
#define GBM_RING_TABLE(NAME, EPI) GBX_TILES(GBM_KERNEL_, 0, EPI) GBX_TILES(GBM_KERNEL_, 1, EPI)
#define GBM_PART_TABLE(NAME) GBX_TILES(GBM_KERNEL_, 0, EPI_PART)
#else
#define GBM_RING_TABLE(NAME, EPI) \
    const gbm::LaunchFn gbm::NAME[2][gbm::kTiles] = {{GBX_TILES(GBM_LAUNCH_, 0, EPI)}, {GBX_TILES(GBM_LAUNCH_, 1, EPI)}};
#define GBM_PART_TABLE(NAME) const gbm::LaunchFn gbm::NAME[gbm::kTiles] = {GBX_TILES(GBM_LAUNCH_, 0, EPI_PART)};
#endif
