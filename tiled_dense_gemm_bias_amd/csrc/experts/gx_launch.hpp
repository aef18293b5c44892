// Launchers of the kernel instances: tables of function pointers, one
// translation unit each. The device pass instantiates the kernels, the host pass
// defines the table.
#pragma once

#include "gx_persist.hpp"
#include "gx_ring.hpp"

namespace gbx {

using LaunchFn = hipError_t (*)(Group, hipStream_t);

// Ring kernel tiles: X(columns of the table, BM, BN, WM, WN, STAGES). The stages
// are what lets two to four workgroups share a CU.
#define GBX_TILES(X, ...)                                                                       \
    X(16, 64, 1, 4, 4, __VA_ARGS__) X(32, 64, 1, 4, 4, __VA_ARGS__) X(64, 64, 2, 2, 3, __VA_ARGS__) \
    X(64, 128, 2, 2, 3, __VA_ARGS__) X(128, 64, 2, 2, 2, __VA_ARGS__) X(128, 128, 2, 2, 2, __VA_ARGS__)
enum { TILE_16x64, TILE_32x64, TILE_64x64, TILE_64x128, TILE_128x64, TILE_128x128, kTiles };
// Weight gradients (At's swizzle needs 64 rows).
#define GBX_GRAD_TILES(X, ...) X(64, 64, 2, 2, 4, __VA_ARGS__) X(128, 128, 2, 2, 2, __VA_ARGS__)
enum { GRAD_64x64, GRAD_128x128, kGradTiles };

// [operand type: f16, bf16][tile]; part_*: partial sums of a split.
extern const LaunchFn fwd_nt[2][kTiles], part_nt[2][kTiles];      // B [N][K]
extern const LaunchFn fwd_nn[2][kTiles], part_nn[2][kTiles];      // B [K][N]
extern const LaunchFn slope_nt[2][kTiles], slope_nn[2][kTiles];
extern const LaunchFn wgrad_tn[2][kGradTiles], part_tn[2][kGradTiles];
extern const LaunchFn mx4_nt[2][kTiles];                          // [output type]
extern const LaunchFn part_mx4[2][kTiles];                        // both the same

// Persistent 256 x 256 kernels: [act], one table an operand type.
extern const LaunchFn big_fwd_nt_f16[kNumActs], big_fwd_nt_bf16[kNumActs];
extern const LaunchFn big_fwd_nn_f16[kNumActs], big_fwd_nn_bf16[kNumActs];
extern const LaunchFn big_slope_nt_f16[kNumActs], big_slope_nt_bf16[kNumActs];
extern const LaunchFn big_slope_nn_f16[kNumActs], big_slope_nn_bf16[kNumActs];
extern const LaunchFn big_mx4_f16[kNumActs], big_mx4_bf16[kNumActs];   // by the output's type
extern const LaunchFn big_wgrad_tn[2][kNumGrads];   // [operand type][GRAD_*]

}  // namespace gbx

#define GBX_KERNEL_(BM, BN, WM, WN, ST, OP, DT, EPI, TB, TA) \
    template __global__ void gbx::grouped_ring_kernel<BM, BN, WM, WN, ST, OP, DT, gbx::EPI, TB, TA>(gbx::Group);
#define GBX_LAUNCH_(BM, BN, WM, WN, ST, OP, DT, EPI, TB, TA) gbx::launch_ring<BM, BN, WM, WN, ST, OP, DT, gbx::EPI, TB, TA>,
#ifdef __HIP_DEVICE_COMPILE__
#define GBX_TABLE_(NAME, N, TILES, O0, O1, T0, T1, ...) TILES(GBX_KERNEL_, O0, T0, __VA_ARGS__) TILES(GBX_KERNEL_, O1, T1, __VA_ARGS__)
#define GBX_MX4_PART_TABLE(NAME) GBX_TILES(GBX_KERNEL_, 2, 0, EPI_PART, true, false)
#else
#define GBX_TABLE_(NAME, N, TILES, O0, O1, T0, T1, ...) \
    const gbx::LaunchFn gbx::NAME[2][gbx::N] = {{TILES(GBX_LAUNCH_, O0, T0, __VA_ARGS__)}, {TILES(GBX_LAUNCH_, O1, T1, __VA_ARGS__)}};
#define GBX_MX4_PART_TABLE(NAME)                                                                \
    const gbx::LaunchFn gbx::NAME[2][gbx::kTiles] = {{GBX_TILES(GBX_LAUNCH_, 2, 0, EPI_PART, true, false)}, \
                                                     {GBX_TILES(GBX_LAUNCH_, 2, 0, EPI_PART, true, false)}};
#endif
// 16-bit operands (the output's type is theirs), weight gradients, 4-bit operands with each output type.
#define GBX_RING_TABLE(NAME, EPI, TB) GBX_TABLE_(NAME, kTiles, GBX_TILES, 0, 1, 0, 1, EPI, TB, false)
#define GBX_GRAD_TABLE(NAME, EPI) GBX_TABLE_(NAME, kGradTiles, GBX_GRAD_TILES, 0, 1, 0, 1, EPI, false, true)
#define GBX_MX4_TABLE(NAME) GBX_TABLE_(NAME, kTiles, GBX_TILES, 2, 2, 0, 1, EPI_ACT, true, false)

#define GBX_BIG_KERNEL_(...) template __global__ void gbx::grouped_persist_kernel<__VA_ARGS__>(gbx::Group);
#ifdef __HIP_DEVICE_COMPILE__
#define GBX_BIG_TABLE(NAME, OP, DT, EPI, TB)                                                    \
    GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 0, TB, false) GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 1, TB, false) \
    GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 2, TB, false) GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 3, TB, false) \
    GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 4, TB, false) GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 5, TB, false)
#define GBX_BIG_WGRAD_(T)                                                                       \
    GBX_BIG_KERNEL_(T, T, gbx::EPI_GRAD, 0, false, true) GBX_BIG_KERNEL_(T, T, gbx::EPI_GRAD, 1, false, true) \
    GBX_BIG_KERNEL_(T, T, gbx::EPI_GRAD, 2, false, true) GBX_BIG_KERNEL_(T, T, gbx::EPI_GRAD, 3, false, true) \
    GBX_BIG_KERNEL_(T, T, gbx::EPI_GRAD, 4, false, true) GBX_BIG_KERNEL_(T, T, gbx::EPI_GRAD, 5, false, true)
#define GBX_BIG_WGRAD_TABLE(NAME) GBX_BIG_WGRAD_(0) GBX_BIG_WGRAD_(1)
#else
#define GBX_BIG_TABLE(NAME, OP, DT, EPI, TB)                                                    \
    const gbx::LaunchFn gbx::NAME[gba::kNumActs] = {                                            \
        gbx::launch_persist<OP, DT, gbx::EPI, 0, TB, false>, gbx::launch_persist<OP, DT, gbx::EPI, 1, TB, false>, \
        gbx::launch_persist<OP, DT, gbx::EPI, 2, TB, false>, gbx::launch_persist<OP, DT, gbx::EPI, 3, TB, false>, \
        gbx::launch_persist<OP, DT, gbx::EPI, 4, TB, false>, gbx::launch_persist<OP, DT, gbx::EPI, 5, TB, false>};
#define GBX_BIG_WGRAD_(T)                                                                       \
    {gbx::launch_persist<T, T, gbx::EPI_GRAD, 0, false, true>, gbx::launch_persist<T, T, gbx::EPI_GRAD, 1, false, true>, \
     gbx::launch_persist<T, T, gbx::EPI_GRAD, 2, false, true>, gbx::launch_persist<T, T, gbx::EPI_GRAD, 3, false, true>, \
     gbx::launch_persist<T, T, gbx::EPI_GRAD, 4, false, true>, gbx::launch_persist<T, T, gbx::EPI_GRAD, 5, false, true>}
#define GBX_BIG_WGRAD_TABLE(NAME) const gbx::LaunchFn gbx::NAME[2][gbx::kNumGrads] = {GBX_BIG_WGRAD_(0), GBX_BIG_WGRAD_(1)};
#endif
