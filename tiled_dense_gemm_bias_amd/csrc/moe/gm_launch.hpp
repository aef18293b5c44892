// Tables of the products' kernel instances, one translation unit each (the device pass instantiates
// the kernels, the host pass defines the table). Tiles as gx_launch.hpp's.
#pragma once

#include "../experts/gx_launch.hpp"
#include "gm_persist.hpp"
#include "gm_stream.hpp"

namespace gbm {

using gbx::Group;
using gbx::kTiles;
using gbx::LaunchFn;

extern const LaunchFn f8_act[2][kTiles], f8_slope[2][kTiles];   // [output type][tile]
extern const LaunchFn f8_part[kTiles];
extern const LaunchFn f8_stream_act[2], f8_stream_slope[2];   // [output type]
// Persistent 256 x 256 kernels: [act], one table an output type.
extern const LaunchFn big_f8_act_f16[kNumActs], big_f8_act_bf16[kNumActs], big_f8_slope_f16[kNumActs], big_f8_slope_bf16[kNumActs];

}  // namespace gbm

#define GBM_KERNEL_(BM, BN, WM, WN, ST, DT, EPI) \
    template __global__ void gbx::grouped_ring_kernel<BM, BN, WM, WN, ST, gbx::OP_F8, DT, gbx::EPI, true, false>(gbx::Group);
#define GBM_LAUNCH_(BM, BN, WM, WN, ST, DT, EPI) gbx::launch_ring<BM, BN, WM, WN, ST, gbx::OP_F8, DT, gbx::EPI, true, false>,
#define GBM_BIG_KERNEL_(DT, EPI, ACT) template __global__ void gbm::f8_persist_kernel<DT, gbx::EPI, ACT>(gbx::Group);
#define GBM_BIG_LAUNCH_(DT, EPI, ACT) gbm::launch_f8_persist<DT, gbx::EPI, ACT>,
#define GBM_BIG_ACTS_(X, DT, EPI) X(DT, EPI, 0) X(DT, EPI, 1) X(DT, EPI, 2) X(DT, EPI, 3) X(DT, EPI, 4) X(DT, EPI, 5)
#ifdef __HIP_DEVICE_COMPILE__
#define GBM_STREAM_TABLE(NAME, EPI) \
    template __global__ void gbm::f8_stream_kernel<0, gbx::EPI>(gbx::Group); template __global__ void gbm::f8_stream_kernel<1, gbx::EPI>(gbx::Group);
#define GBM_BIG_TABLE(NAME, DT, EPI) GBM_BIG_ACTS_(GBM_BIG_KERNEL_, DT, EPI)
#define GBM_RING_TABLE(NAME, EPI) GBX_TILES(GBM_KERNEL_, 0, EPI) GBX_TILES(GBM_KERNEL_, 1, EPI)
#define GBM_PART_TABLE(NAME) GBX_TILES(GBM_KERNEL_, 0, EPI_PART)
#else
#define GBM_STREAM_TABLE(NAME, EPI) \
    const gbm::LaunchFn gbm::NAME[2] = {gbm::launch_f8_stream<0, gbx::EPI>, gbm::launch_f8_stream<1, gbx::EPI>};
#define GBM_BIG_TABLE(NAME, DT, EPI) const gbm::LaunchFn gbm::NAME[gba::kNumActs] = {GBM_BIG_ACTS_(GBM_BIG_LAUNCH_, DT, EPI)};
#define GBM_RING_TABLE(NAME, EPI) \
    const gbm::LaunchFn gbm::NAME[2][gbm::kTiles] = {{GBX_TILES(GBM_LAUNCH_, 0, EPI)}, {GBX_TILES(GBM_LAUNCH_, 1, EPI)}};
#define GBM_PART_TABLE(NAME) const gbm::LaunchFn gbm::NAME[gbm::kTiles] = {GBX_TILES(GBM_LAUNCH_, 0, EPI_PART)};
#endif
