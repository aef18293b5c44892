// Column sums of each expert's rows (bias gradients beside the ring kernel). Bound by
// HBM, dC read once, where there are about as many column blocks as CUs (16384 x 8192 by 8
// experts: 43 us, 6.2 TB/s); few long experts by a workgroup's walk along the rows, which are
// not split (16384 x 1024, one expert, 16 workgroups: 23 us, 1.4 TB/s).
#pragma once

#include "gx_common.hpp"

namespace gbx {

// A workgroup sums COLS columns of one expert in fp32: COLS / 8 lanes of eight
// columns by RL row lanes that stride over the rows, joined in a fixed order.
template <int DT, int COLS, int NT>
__global__ void __launch_bounds__(NT)
column_sums_kernel(Group g) {
    constexpr int CL = COLS / 8, RL = NT / CL;
    __shared__ float part[RL][COLS];
    const int col = threadIdx.x % CL, lane_row = threadIdx.x / CL;
    const int n = blockIdx.x * COLS + col * 8;
    const int e = blockIdx.y;
    int start, rows;
    expert_rows(g, e, start, rows);
    float sum[8] = {};
    if (n < g.N) {
        const uint16_t *const p = g.A + (size_t)start * g.N + n;
#pragma unroll 4
        for (int r = lane_row; r < rows; r += RL) {
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
    // Halves are joined until one row is left.
#pragma unroll
    for (int h = RL / 2; h >= 1; h /= 2) {
        __syncthreads();
        for (int i = threadIdx.x; i < h * COLS; i += NT) part[i / COLS][i % COLS] += part[i / COLS + h][i % COLS];
    }
    __syncthreads();
    const int c = threadIdx.x * 2, nc = blockIdx.x * COLS + c;
    if (c >= COLS || nc >= g.N) return;   // N is a multiple of 8
    const float a = part[0][c], b = part[0][c + 1];
    const size_t at = (size_t)e * g.N + nc;
    if (g.flags & GF_F32) {
        float *const o = (float *)g.C + at;
        o[0] = (g.flags & GF_ADD) ? o[0] + a : a;
        o[1] = (g.flags & GF_ADD) ? o[1] + b : b;
    } else {
        *reinterpret_cast<uint32_t *>((uint16_t *)g.C + at) = pack2<DT>(a, b);
    }
}

template <int DT, int COLS, int NT>
hipError_t launch_sums(const Group &g, hipStream_t stream) {
    return launch(column_sums_kernel<DT, COLS, NT>, dim3((unsigned)ceil_div(g.N, COLS), (unsigned)g.E), dim3(NT), stream, g);
}

// 64 columns are a 128-byte line of a row. Long experts take eight waves, so that
// more rows are on their way at once: 16384 x 1024 (one expert) 23 us, with four
// waves 36, sixteen 19; 64 experts of 32 rows x 2816 the other way round: 6.9, 5.4 and 12 us.
inline hipError_t launch_column_sums(const Group &g, int dtype, hipStream_t stream) {
    const bool f16 = dtype == DT_F16, wide = g.T / g.E >= 512;
    if (wide) return f16 ? launch_sums<DT_F16, 64, 512>(g, stream) : launch_sums<DT_BF16, 64, 512>(g, stream);
    return f16 ? launch_sums<DT_F16, 64, 256>(g, stream) : launch_sums<DT_BF16, 64, 256>(g, stream);
}

}  // namespace gbx
