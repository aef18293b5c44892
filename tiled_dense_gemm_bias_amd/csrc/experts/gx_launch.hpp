// Launchers of the kernel instances: tables of function pointers, one
// translation unit each. The device pass instantiates the kernels, the host pass
// defines the table.
#pragma once

#include "gx_persist.hpp"
#include "gx_ring.hpp"

namespace gbx {

using LaunchFn = hipError_t (*)(Group, hipStream_t);
enum { TILE_16x64 = 0, TILE_64x64 = 1, TILE_128x128 = 2, kTiles = 3 };

// [operand type: f16, bf16][tile]
extern const LaunchFn fwd_nt[2][kTiles];      // B [N][K]
extern const LaunchFn fwd_nn[2][kTiles];      // B [K][N]
extern const LaunchFn slope_nt[2][kTiles];
extern const LaunchFn slope_nn[2][kTiles];
extern const LaunchFn wgrad_tn[2][kTiles];    // no 16x64 tile: At's swizzle needs 64 rows
extern const LaunchFn mx4_nt[2][kTiles];      // [output type]

// Persistent 256 x 256 kernels: [act], one table an operand type.
extern const LaunchFn big_fwd_nt_f16[kNumActs], big_fwd_nt_bf16[kNumActs];
extern const LaunchFn big_fwd_nn_f16[kNumActs], big_fwd_nn_bf16[kNumActs];
extern const LaunchFn big_slope_nt_f16[kNumActs], big_slope_nt_bf16[kNumActs];
extern const LaunchFn big_slope_nn_f16[kNumActs], big_slope_nn_bf16[kNumActs];
extern const LaunchFn big_mx4_f16[kNumActs], big_mx4_bf16[kNumActs];   // by the output's type
extern const LaunchFn big_wgrad_tn[2][2];   // [operand type][GRAD_16, GRAD_F32]

}  // namespace gbx

#define GBX_RING_KERNEL_(...) template __global__ void gbx::grouped_ring_kernel<__VA_ARGS__>(gbx::Group);
#ifdef __HIP_DEVICE_COMPILE__
#define GBX_RING_TABLE_(NAME, O0, O1, T0, T1, EPI, TB)                                          \
    GBX_RING_KERNEL_(16, 64, 1, 4, 4, O0, T0, EPI, TB, false)                                   \
    GBX_RING_KERNEL_(64, 64, 2, 2, 4, O0, T0, EPI, TB, false)                                   \
    GBX_RING_KERNEL_(128, 128, 2, 2, 2, O0, T0, EPI, TB, false)                                 \
    GBX_RING_KERNEL_(16, 64, 1, 4, 4, O1, T1, EPI, TB, false)                                   \
    GBX_RING_KERNEL_(64, 64, 2, 2, 4, O1, T1, EPI, TB, false)                                   \
    GBX_RING_KERNEL_(128, 128, 2, 2, 2, O1, T1, EPI, TB, false)
#define GBX_RING_WGRAD_TABLE(NAME)                                                              \
    GBX_RING_KERNEL_(64, 64, 2, 2, 4, 0, 0, gbx::EPI_GRAD, false, true)                         \
    GBX_RING_KERNEL_(128, 128, 2, 2, 2, 0, 0, gbx::EPI_GRAD, false, true)                       \
    GBX_RING_KERNEL_(64, 64, 2, 2, 4, 1, 1, gbx::EPI_GRAD, false, true)                         \
    GBX_RING_KERNEL_(128, 128, 2, 2, 2, 1, 1, gbx::EPI_GRAD, false, true)
#else
#define GBX_RING_TABLE_(NAME, O0, O1, T0, T1, EPI, TB)                                          \
    const gbx::LaunchFn gbx::NAME[2][gbx::kTiles] = {                                           \
        {gbx::launch_ring<16, 64, 1, 4, 4, O0, T0, EPI, TB, false>,                             \
         gbx::launch_ring<64, 64, 2, 2, 4, O0, T0, EPI, TB, false>,                             \
         gbx::launch_ring<128, 128, 2, 2, 2, O0, T0, EPI, TB, false>},                          \
        {gbx::launch_ring<16, 64, 1, 4, 4, O1, T1, EPI, TB, false>,                             \
         gbx::launch_ring<64, 64, 2, 2, 4, O1, T1, EPI, TB, false>,                             \
         gbx::launch_ring<128, 128, 2, 2, 2, O1, T1, EPI, TB, false>}};
#define GBX_RING_WGRAD_TABLE(NAME)                                                              \
    const gbx::LaunchFn gbx::NAME[2][gbx::kTiles] = {                                           \
        {nullptr, gbx::launch_ring<64, 64, 2, 2, 4, 0, 0, gbx::EPI_GRAD, false, true>,          \
         gbx::launch_ring<128, 128, 2, 2, 2, 0, 0, gbx::EPI_GRAD, false, true>},                \
        {nullptr, gbx::launch_ring<64, 64, 2, 2, 4, 1, 1, gbx::EPI_GRAD, false, true>,          \
         gbx::launch_ring<128, 128, 2, 2, 2, 1, 1, gbx::EPI_GRAD, false, true>}};
#endif
// 16-bit operands (the output's type is theirs), or 4-bit ones with each output type.
#define GBX_RING_TABLE(NAME, EPI, TB) GBX_RING_TABLE_(NAME, 0, 1, 0, 1, gbx::EPI, TB)
#define GBX_RING_MX4_TABLE(NAME) GBX_RING_TABLE_(NAME, 2, 2, 0, 1, gbx::EPI_ACT, true)

#define GBX_BIG_KERNEL_(...) template __global__ void gbx::grouped_persist_kernel<__VA_ARGS__>(gbx::Group);
#ifdef __HIP_DEVICE_COMPILE__
#define GBX_BIG_TABLE(NAME, OP, DT, EPI, TB)                                                    \
    GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 0, TB, false) GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 1, TB, false) \
    GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 2, TB, false) GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 3, TB, false) \
    GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 4, TB, false) GBX_BIG_KERNEL_(OP, DT, gbx::EPI, 5, TB, false)
#define GBX_BIG_WGRAD_TABLE(NAME)                                                               \
    GBX_BIG_KERNEL_(0, 0, gbx::EPI_GRAD, 0, false, true) GBX_BIG_KERNEL_(0, 0, gbx::EPI_GRAD, 1, false, true) \
    GBX_BIG_KERNEL_(1, 1, gbx::EPI_GRAD, 0, false, true) GBX_BIG_KERNEL_(1, 1, gbx::EPI_GRAD, 1, false, true)
#else
#define GBX_BIG_TABLE(NAME, OP, DT, EPI, TB)                                                    \
    const gbx::LaunchFn gbx::NAME[gba::kNumActs] = {                                            \
        gbx::launch_persist<OP, DT, gbx::EPI, 0, TB, false>, gbx::launch_persist<OP, DT, gbx::EPI, 1, TB, false>, \
        gbx::launch_persist<OP, DT, gbx::EPI, 2, TB, false>, gbx::launch_persist<OP, DT, gbx::EPI, 3, TB, false>, \
        gbx::launch_persist<OP, DT, gbx::EPI, 4, TB, false>, gbx::launch_persist<OP, DT, gbx::EPI, 5, TB, false>};
#define GBX_BIG_WGRAD_TABLE(NAME)                                                               \
    const gbx::LaunchFn gbx::NAME[2][2] = {                                                     \
        {gbx::launch_persist<0, 0, gbx::EPI_GRAD, 0, false, true>, gbx::launch_persist<0, 0, gbx::EPI_GRAD, 1, false, true>}, \
        {gbx::launch_persist<1, 1, gbx::EPI_GRAD, 0, false, true>, gbx::launch_persist<1, 1, gbx::EPI_GRAD, 1, false, true>}};
#endif
