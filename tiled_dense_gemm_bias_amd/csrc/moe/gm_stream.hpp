// 8-bit products of few rows an expert: reading the weights once is all there is to do, so nothing of them is staged.
//
// A workgroup takes 16 rows of one expert x 16 columns. Its four waves share the depth, a quarter of the slices each
// (a slice: 128 values, one block, one matrix instruction of 16 columns x 16 rows), and load their operands
// straight into registers in the instruction's layout: lane l has row / column l % 16, 16-byte chunks l / 16 and l / 16
// + 4 of the slice. There is no barrier until the waves' sums are joined through LDS, in wave order. Rows past
// the expert's end are not fetched; those that are there are read again for every 16 columns, so that more than some
// eight of them are the ring kernel's (16 rows of 4096 x 14336: 17.6 us, ring 14.9).
//
// What bounds it: HBM, and the start of a kernel: 8 rows on 8 experts of 4096 x 4096 take 26.2 us (5.1 TB/s, as a large
// copy; ring 29.6), 16 rows on 12 of 32 experts of 2816 x 2048 15.8 (4.4 TB/s; ring 16.7), 1 x 4096 x 4096 7.1 (ring 8.8). Two
// slices' loads at a time and eight workgroups a CU: with four and five 16.4 us, as the start and the end of a
// workgroup are then less covered. Sixteen waves a workgroup gain only where there are few columns (1 x 1024 x 8192 9.6
// -> 8.5 us, 2816 x 2048 15.8 -> 26.2). Non-temporal loads take 18.0: the two halves of a line come by two
// instructions, and it is fetched twice.
#pragma once

#include "gm_common.hpp"

namespace gbm {

using gbx::Found;
using gbx::Group;

template <int ODT, int EPI>
__global__ void __launch_bounds__(256, 8)   // eight waves a SIMD
f8_stream_kernel(Group g) {
    constexpr int BM = 16, BN = 16, WAVES = 4, BATCH = 2;
    __shared__ __attribute__((aligned(16))) float sums[WAVES][BM][BN + 4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tg = lane >> 4, tj = lane & 15;

    // ---- the work unit ----
    const int tiles_n = ceil_div(g.N, BN);
    const long long b = (long long)blockIdx.y * gridDim.x + blockIdx.x;
    int u = -1;
    Found f;
    auto row_tile = [&](int total) __attribute__((always_inline)) {
        u = b < (long long)total * tiles_n ? (int)b : -1;
        return u < 0 ? -1 : u / tiles_n;
    };
    if (g.E <= 64) {
        f = gbx::locate_few(g, BM, lane, row_tile);
        if (u < 0) return;
    } else {
        const int t = row_tile(gbx::total_row_tiles(g, BM, lane));
        if (u < 0) return;
        f = gbx::find_row_tile(g, BM, t, lane);
    }
    const int m0 = (u / tiles_n - f.before) * BM, n0 = u % tiles_n * BN;
    // Offsets that decrease could name a tile past its expert's rows.
    if (m0 < 0 || m0 >= f.rows) return;
    const int rows = min(f.rows - m0, BM), cols = min(g.N - n0, BN);
    const uint32_t KB = (uint32_t)g.K * 2u;   // bytes (values) of a row
    const int nk = ceil_div(g.K, 64);
    const int k0 = (int)((long long)wid * nk / WAVES), k1 = (int)((long long)(wid + 1) * nk / WAVES);

    // 16 rows of at most 2^22 bytes: offsets below 2^31.
    const __amdgpu_buffer_rsrc_t ra = make_rsrc((const char *)g.A + (size_t)(f.start + m0) * KB, (uint32_t)rows * KB);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc((const char *)g.B + ((size_t)f.e * g.N + n0) * KB, (uint32_t)cols * KB);
    typedef const float __attribute__((address_space(4))) *ScalePtr;
    const ScalePtr sw = (ScalePtr)(uintptr_t)((const float *)g.sb + ((size_t)f.e * ceil_div(g.N, 128) + n0 / 128) * nk);
    const float *const sa = (const float *)g.sa + f.start + m0;

    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int k = k0; k < k1; k += BATCH) {
        u32x4 w[BATCH][2], a[BATCH][2];
        float s[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const bool there = k + i < k1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = (uint32_t)(k + i) * 128u + (uint32_t)(tg + 4 * h) * 16u;
                const uint32_t off = there && at < KB ? (uint32_t)tj * KB + at : kOobOffset;
                w[i][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, (int)off, 0, 0));
                a[i][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, (int)off, 0, 0));
            }
            s[i] = 0.0f;
            if (there && tj < rows) s[i] = sa[(size_t)(k + i) * g.T + tj];
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (k + i >= k1) continue;
            auto both = [](const u32x4 (&x)[2]) __attribute__((always_inline)) {
                return gbx::i32x8{(int)x[0].x, (int)x[0].y, (int)x[0].z, (int)x[0].w, (int)x[1].x, (int)x[1].y, (int)x[1].z, (int)x[1].w};
            };
            const f32x4 p = gbx::mfma_f8(both(w[i]), both(a[i]));
            const float by = s[i] * sw[k + i];
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = fmaf(p[q], by, acc[q]);
        }
    }
    *reinterpret_cast<f32x4 *>(&sums[wid][tj][4 * tg]) = acc;
    __syncthreads();
    // Thread: eight columns of one row.
    const int r = tid >> 1, c = (tid & 1) * 8;
    if (r >= rows || c >= cols) return;   // (N is a multiple of 8)
    f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int q = 0; q < WAVES; ++q) {
        v[0] += *reinterpret_cast<const f32x4 *>(&sums[q][r][c]);
        v[1] += *reinterpret_cast<const f32x4 *>(&sums[q][r][c + 4]);
    }
    gbx::finish<EPI, ODT>(g, v, f.e, n0 + c, (size_t)(f.start + m0 + r) * g.N + n0 + c);
}

template <int ODT, int EPI>
hipError_t launch_f8_stream(Group g, hipStream_t stream) {
    const long long row_tiles = gbx::row_tile_bound(g.T, g.E, 16), units = row_tiles * ceil_div(g.N, 16);
    if (units <= 0) return hipSuccess;
    if (units > 0x7fffffffLL - kGridX) return hipErrorInvalidValue;
    g.row_bound = (int)row_tiles;
    return launch(f8_stream_kernel<ODT, EPI>, tile_grid(units), dim3(256), stream, g);
}

}  // namespace gbm
