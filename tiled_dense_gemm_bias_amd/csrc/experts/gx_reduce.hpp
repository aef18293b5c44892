// Second pass of a split sum, bound by its launch where splits pay (16 x 2816 of four
// splits: 4.4 us): adds the splits' fp32 partial sums in split order
// (the result does not depend on which was written first), then the epilogue.
#pragma once

#include "gx_common.hpp"

namespace gbx {

// A wave takes 512 columns of one row, eight a lane; a workgroup four rows. P:
// [splits][rows][N]. Rows mode: rows of no expert have no sums and are left alone.
template <int EPI, int ODT, bool TA>
__global__ void __launch_bounds__(256)
grouped_reduce_kernel(Group g) {
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const long long rows = TA ? (long long)g.E * g.M : (long long)g.T;
    const long long row = ((long long)blockIdx.y * gridDim.z + blockIdx.z) * 4 + wid;
    if (row >= rows) return;
    int e = 0;
    if (!TA && g.offsets) {
        unsigned long long mine = 0;
        for (int e0 = 0; e0 < g.E && !mine; e0 += 64) {
            bool in = false;
            if (e0 + lane < g.E) {
                int start, n;
                expert_rows(g, e0 + lane, start, n);
                in = row >= start && row < (long long)start + n;
            }
            mine = __ballot(in);
            if (mine) e = e0 + __ffsll(mine) - 1;
        }
        if (!mine) return;
    }
    const int n = blockIdx.x * 512 + lane * 8;
    if (n >= g.N) return;
    const size_t at = (size_t)row * g.N + n, plane = (size_t)rows * g.N;
    f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
        const f32x4 *const p = reinterpret_cast<const f32x4 *>(g.part + s * plane + at);
        v[0] += __builtin_nontemporal_load(p);
        v[1] += __builtin_nontemporal_load(p + 1);
    }
    finish<EPI, ODT>(g, v, e, n, at);
}

template <int EPI, int ODT, bool TA>
hipError_t launch_reduce(Group g, hipStream_t stream) {
    const long long rows = TA ? (long long)g.E * g.M : (long long)g.T, groups = (rows + 3) / 4;
    const long long z = groups < 32768 ? 1 : (groups + 32767) / 32768;   // grid dimensions of at most 2^16
    const dim3 grid((unsigned)ceil_div(g.N, 512), (unsigned)((groups + z - 1) / z), (unsigned)z);
    return launch(grouped_reduce_kernel<EPI, ODT, TA>, grid, dim3(256), stream, g);
}

}  // namespace gbx
