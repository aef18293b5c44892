// Movement of rows between tokens and experts. rows[t][j] is the row of slot (t, j), or -1; a
// number outside [0, R) counts as -1.
//
//   dispatch:      out[rows[t][j]] = x[t]
//   combine:       out[t] = sum_j w[t][j] y[rows[t][j]], in 32 bits in the order of j
//   combine_grad:  dy[rows[t][j]] = w[t][j] dout[t], dw[t][j] = <dout[t], y[rows[t][j]]>
//
// HBM is what bounds them: every row is read and written once (a token's x and dout once for its k slots). 8192 tokens of
// 4096 and 4 slots each: dispatch 53 us (6.3 TB/s; a large copy runs at 5.1), combine 59 (5.7), combine_grad 103 (5.8).
// A workgroup takes one token and up to 8 KiB of its row: eight values a lane and load, a
// token's loads all out before the first is used.
#pragma once

#include "gm_common.hpp"

namespace gbm {

struct Move {
    const void *x;             // tokens' rows [T][H] (F32: in 32 bits)
    const uint16_t *y;         // experts' rows [R][H]
    const int32_t *rows;       // [T][k]
    const float *w;            // [T][k] or null (ones)
    void *out;                 // as x
    uint16_t *dy;
    float *dw;                 // [T][k] or null
    int T, k, H, R;
};

constexpr int kMoveThreads = 256;

__device__ __forceinline__ long long move_token() { return (long long)blockIdx.z * gridDim.y + blockIdx.y; }

// Grid: pieces of a row along x, tokens along y and z.
inline dim3 move_grid(long long tokens, int pieces) {
    const long long z = (tokens + 32767) / 32768;
    return dim3((unsigned)pieces, (unsigned)((tokens + z - 1) / z), (unsigned)z);
}

__global__ void __launch_bounds__(kMoveThreads)
dispatch_kernel(Move a) {
    const long long t = move_token();
    const int h = (blockIdx.x * kMoveThreads + threadIdx.x) * 8;
    if (t >= a.T || h >= a.H) return;
    const u32x4 v = *reinterpret_cast<const u32x4 *>((const uint16_t *)a.x + (size_t)t * a.H + h);
    const int32_t *const rows = a.rows + (size_t)t * a.k;
    for (int j = 0; j < a.k; ++j) {
        const int r = rows[j];
        if ((unsigned)r < (unsigned)a.R) __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>((uint16_t *)a.out + (size_t)r * a.H + h));
    }
}

template <int DT>
__device__ __forceinline__ void unpack8(const u32x4 &x, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = to_f32<DT>(x[i] & 0xffffu);
        v[2 * i + 1] = to_f32<DT>(x[i] >> 16);
    }
}
template <int DT>
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
    return u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
}

// F32: the sums leave as they are, where a caller's own arithmetic on them (a loss, say) is in 32 bits.
template <int DT, bool F32>
__global__ void __launch_bounds__(kMoveThreads)
combine_kernel(Move a) {
    const long long t = move_token();
    const int h = (blockIdx.x * kMoveThreads + threadIdx.x) * 8;
    if (t >= a.T || h >= a.H) return;
    const int32_t *const rows = a.rows + (size_t)t * a.k;
    float sum[8] = {};
    constexpr int N = 8;
    for (int j0 = 0; j0 < a.k; j0 += N) {
        u32x4 v[N];
        float w[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int r = j0 + j < a.k ? rows[j0 + j] : -1;
            const bool there = (unsigned)r < (unsigned)a.R;
            v[j] = u32x4{0u, 0u, 0u, 0u};
            if (there) v[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(a.y + (size_t)r * a.H + h));
            // A slot without a row adds w 0: a weight of NaN shows.
            w[j] = j0 + j >= a.k ? 0.0f : a.w ? a.w[(size_t)t * a.k + j0 + j] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float f[8];
            unpack8<DT>(v[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[j], f[i], sum[i]);
        }
    }
    const size_t at = (size_t)t * a.H + h;
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __builtin_nontemporal_store(f32x4{sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]},
                                        reinterpret_cast<f32x4 *>((float *)a.out + at + 4 * i));
    } else {
        __builtin_nontemporal_store(pack8<DT>(sum), reinterpret_cast<u32x4 *>((uint16_t *)a.out + at));
    }
}

constexpr int kGradPieces = 4, kMaxSlots = 32;   // pieces of eight columns that a thread holds of dout at a time

// W waves a token, 4 / W tokens a workgroup. Where tokens are many and their rows short of 4096 one wave a token is faster, as
// all its lanes have columns (4 slots, a wave and four: 65536 x 512 132 and 403 us, 32768 x 1024 110 and 242, 16384 x 2048 114
// and 150, 8192 x 2816 82 and 88, 8192 x 4096 114 both, 8192 x 7168 200 and 193); few tokens want more waves each, and the fewer
// the columns the earlier they have enough: 4 slots, a wave and four: of 128 columns 512 tokens 5.6 and 5.8, 1500 6.3 and 10.2; 1024
// columns 256 7.0 and 6.8, 512 8.0 both, 1500 10.3 and 15.5; 2048 columns 1000 13.0 and 11.8, 1500 15.1 and 18.3; 2816 columns 1500
// 23.5 and 21.1, 2048 26.5 and 24.8, 2500 30.0 and 31.4; 3584 columns 2048 28.9 and 28.4, 3000 38.5 and 39.8. (With 1, 2 and 8
// slots the same within 10 %: 8 slots of 1024 columns 512 13.9 and 13.7, 768 14.9 and 15.4; 2048 columns 1000 23.3 and 19.7, 1200 25.4
// and 29.6; 1 slot of 2816 2048 10.2 both.) The next slot's row loaded ahead took longer everywhere (16384 x 2048 115; twice
// the registers).
inline bool one_wave_a_token(long long T, int H) { return T > (H <= 1024 ? 512 : H <= 2048 ? 1024 : 2304) && H < 4096; }

// F32: dout as combine's sums, in 32 bits.
template <int DT, int W, bool F32>
__global__ void __launch_bounds__(kMoveThreads)
combine_grad_kernel(Move a) {
    constexpr int THREADS = 64 * W, COLUMNS = THREADS * 8 * kGradPieces;
    __shared__ float dots[kMoveThreads / 64][kMaxSlots];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, tid = threadIdx.x & (THREADS - 1);
    const long long t = move_token() * (4 / W) + wid / W;
    if (t >= a.T) return;   // all of a token's waves
    const int32_t *const rows = a.rows + (size_t)t * a.k;
    for (int j = lane; j < kMaxSlots; j += 64) dots[wid][j] = 0.0f;
    wave_sync();
    for (int h0 = 0; h0 < a.H; h0 += COLUMNS) {
        float d[kGradPieces][8];
#pragma unroll
        for (int p = 0; p < kGradPieces; ++p) {
            const int h = h0 + (p * THREADS + tid) * 8;
            const size_t at = (size_t)t * a.H + h;
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f32x4 v = {0.f, 0.f, 0.f, 0.f};
                    if (h < a.H) v = *reinterpret_cast<const f32x4 *>((const float *)a.x + at + 4 * i);
#pragma unroll
                    for (int q = 0; q < 4; ++q) d[p][4 * i + q] = v[q];
                }
            } else {
                u32x4 v = {0u, 0u, 0u, 0u};
                if (h < a.H) v = *reinterpret_cast<const u32x4 *>((const uint16_t *)a.x + at);
                unpack8<DT>(v, d[p]);
            }
        }
        for (int j = 0; j < a.k; ++j) {
            const int r = rows[j];
            if ((unsigned)r >= (unsigned)a.R) continue;
            const float w = a.w ? a.w[(size_t)t * a.k + j] : 1.0f;
            u32x4 v[kGradPieces];
#pragma unroll
            for (int p = 0; p < kGradPieces; ++p) {
                const int h = h0 + (p * THREADS + tid) * 8;
                v[p] = u32x4{0u, 0u, 0u, 0u};
                if (h < a.H) v[p] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(a.y + (size_t)r * a.H + h));
            }
            float dot = 0.0f;
#pragma unroll
            for (int p = 0; p < kGradPieces; ++p) {
                const int h = h0 + (p * THREADS + tid) * 8;
                float f[8], o[8];
                unpack8<DT>(v[p], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot = fmaf(d[p][i], f[i], dot);
                    o[i] = w * d[p][i];
                }
                if (a.dy && h < a.H) __builtin_nontemporal_store(pack8<DT>(o), reinterpret_cast<u32x4 *>(a.dy + (size_t)r * a.H + h));
            }
#pragma unroll
            for (int s = 1; s < 64; s *= 2) dot += __shfl_xor(dot, s);
            if (lane == 0) dots[wid][j] += dot;
        }
    }
    if constexpr (W > 1)
        __syncthreads();
    else
        wave_sync();
    if (a.dw && tid < a.k) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += dots[wid / W * W + w][tid];
        a.dw[(size_t)t * a.k + tid] = s;
    }
}

}  // namespace gbm
