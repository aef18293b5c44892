// Column sums of each expert's rows (bias gradients).
#pragma once

#include "gx_common.hpp"

namespace gbx {

// One workgroup sums 128 columns of one expert: 16 lanes of 8 columns by 16 row
// lanes, fp32, joined over the row lanes in a fixed order.
template <int DT>
__global__ void __launch_bounds__(256)
column_sums_kernel(Group g) {
    __shared__ float part[16][128];
    const int col = threadIdx.x & 15, lane_row = threadIdx.x >> 4;
    const int n = blockIdx.x * 128 + col * 8;
    const int e = blockIdx.y;
    int start, rows;
    expert_rows(g, e, start, rows);
    float sum[8] = {};
    if (n < g.N) {
        const uint16_t *const p = g.A + (size_t)start * g.N + n;
#pragma unroll 4
        for (int r = lane_row; r < rows; r += 16) {
            const u32x4 x = *reinterpret_cast<const u32x4 *>(p + (size_t)r * g.N);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[2 * i] += to_f32<DT>(x[i] & 0xffffu);
                sum[2 * i + 1] += to_f32<DT>(x[i] >> 16);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[lane_row][col * 8 + i] = sum[i];
    __syncthreads();
    const int c = threadIdx.x * 2, nc = blockIdx.x * 128 + c;
    if (c >= 128 || nc >= g.N) return;   // N is a multiple of 8
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        a += part[r][c];
        b += part[r][c + 1];
    }
    const size_t at = (size_t)e * g.N + nc;
    if (g.flags & GF_F32) {
        float *const o = (float *)g.C + at;
        o[0] = (g.flags & GF_ADD) ? o[0] + a : a;
        o[1] = (g.flags & GF_ADD) ? o[1] + b : b;
    } else {
        *reinterpret_cast<uint32_t *>((uint16_t *)g.C + at) = pack2<DT>(a, b);
    }
}

inline hipError_t launch_column_sums(const Group &g, int dtype, hipStream_t stream) {
    const dim3 grid((unsigned)ceil_div(g.N, 128), (unsigned)g.E);
    auto *const kernel = dtype == DT_F16 ? column_sums_kernel<DT_F16> : column_sums_kernel<DT_BF16>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, g);
    return hipGetLastError();
}

}  // namespace gbx
