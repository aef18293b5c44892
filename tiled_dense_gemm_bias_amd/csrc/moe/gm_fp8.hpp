// 8-bit floats (OCP E4M3) with one fp32 scale a block of 128, and back.
//
// A block's scale is max / 448 in 32 bits, 2^-126 at least, and a value's code the one nearest to 448 x / max
// (x 2^126 where the scale is 2^-126): the quotient itself, not one by the rounded scale, so that the many x
// on a border between two codes (3/4 of the maximum, say) go to the even one. 448 x / max is
// within 2^-22 of itself when computed as x (448 / max), and either equal to a border or 2^-16 of itself away
// from it (both are quotients of integers of at most 11 and 16 bits): cut to 17 bits it is
// on the right side, or on the border. With powers of two for scales everything is exact.
//
// HBM is what bounds all of these (a large copy runs at 5.1 TB/s): 8 weights of 8192 x 4096 in both layouts 172 us (6.2
// TB/s) and back 134 to 167 each, 32768 rows of 4096 back 65 us (6.2 TB/s).
#pragma once

#include "gm_common.hpp"

namespace gbm {

constexpr float kF8Max = 448.0f, kMinScale = 0x1p-126f;

// Of a block whose largest magnitude is `top`: the scale and what its values are multiplied by. Not finite: NaN
// and 0 (the codes are 0). pow2: the smallest power of two that takes the block in.
__device__ __forceinline__ void block_scale(float top, bool pow2, float &scale, float &by) {
    if (!(top < __builtin_inff())) {
        scale = __builtin_nanf("");
        by = 0.0f;
    } else if (top < kF8Max * kMinScale) {
        scale = kMinScale;
        by = 0x1p126f;
    } else if (pow2) {
        // top / 448 <= 2^j: of top = f 2^e (1 <= f < 2), j is e - 8 for f <= 1.75 and e - 7 above.
        const uint32_t b = __float_as_uint(top);
        const int j = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
        scale = __uint_as_float((uint32_t)(j + 127) << 23);
        by = __uint_as_float((uint32_t)(127 - j) << 23);
    } else {
        scale = top / kF8Max;
        by = kF8Max / top;
    }
}

// x by, cut to 17 bits (see above).
__device__ __forceinline__ float quotient(float x, float by) {
    return __uint_as_float((__float_as_uint(x * by) + 32u) & ~63u);
}

// Eight values to eight codes. `by` 0 (a block that is not finite): zeros.
template <int DT>
__device__ __forceinline__ u32x2 to_f8(const u32x4 &x, float by) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = quotient(to_f32<DT>(x[i] & 0xffffu), by);
        f[2 * i + 1] = quotient(to_f32<DT>(x[i] >> 16), by);
    }
    u32x2 c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
        c[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], v, true);
    }
    return by == 0.0f ? u32x2{0u, 0u} : c;
}

// Eight codes to values times a scale.
template <int DT>
__device__ __forceinline__ u32x4 from_f8(const u32x2 &c, float scale) {
    u32x4 y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
        y[2 * i] = pack2<DT>(a[0] * scale, a[1] * scale);
        y[2 * i + 1] = pack2<DT>(b[0] * scale, b[1] * scale);
    }
    return y;
}

// The largest magnitude's bits of eight 16-bit values (the order of magnitudes is that of their bits; an
// infinity or a NaN is the largest).
__device__ __forceinline__ uint32_t top_bits(const u32x4 &x) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t m = x[i] & 0x7fff7fffu;
        top = max(top, max(m & 0xffffu, m >> 16));
    }
    return top;
}

// The value of the lane N places on among its 16.
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xf, 0xf, true);
}

struct QuantRows {
    const uint16_t *x;        // [T][K]
    const int32_t *rows;      // [T][k], or null: row t goes to row t
    uint8_t *codes;           // [R][K]
    float *scales;            // [blocks of K][R]
    int T, K, k, R;
    int pow2;
};

constexpr int kQuantBlocks = 4;     // a wave: 16 lanes of 8 values a block
constexpr int kDequantRows = 16;    // of a workgroup

// B = 4: a wave takes one row's four blocks: 512 bytes of codes leave together, and the loads of its rows' numbers (a lane each) go
// out with those of the values. 8192 rows of 4096 bf16 to four rows each take 44 us (4.7 TB/s); two rows a wave 47, four 49,
// and four with a row in each 16 lanes, in 128-byte pieces, 50 (8 rows of 2048: 2.7, 2.8, 3.5 and 3.9 us).
// B = 1, 2: rows of no more blocks than that, 4 / B of them a wave (300000 rows of 128: 63 us with B = 4, 24 with 1; 100000 of 384 27).
template <int DT, int B>
__global__ void __launch_bounds__(256)
quantize_rows_kernel(QuantRows a) {
    constexpr int N = kQuantBlocks / B;   // rows a wave
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const long long t = (((long long)blockIdx.z * gridDim.x + blockIdx.x) * 4 + wid) * N + (N == 1 ? 0 : (lane >> 4) / B);
    const int block = blockIdx.y * B + (lane >> 4) % B, c = block * 128 + (lane & 15) * 8;
    if (t >= a.T) return;   // whole rows
    int rows = (int)t;      // N = 1: of slot `lane` (k <= 32); else of slot 0
    if (a.rows) rows = a.rows[(size_t)t * a.k + (N == 1 ? min(lane, a.k - 1) : 0)];
    u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(a.x + (size_t)t * a.K + min(c, a.K - 8)));
    if (c >= a.K) v = u32x4{0u, 0u, 0u, 0u};
    uint32_t top = top_bits(v);
    top = max(top, row_ror<8>(top));
    top = max(top, row_ror<4>(top));
    top = max(top, row_ror<2>(top));
    top = max(top, row_ror<1>(top));
    float scale, by;
    block_scale(to_f32<DT>(top), a.pow2 != 0, scale, by);
    const u32x2 code = to_f8<DT>(v, by);
    for (int j = 0; j < a.k; ++j) {
        int r;
        if constexpr (N == 1) {
            r = __builtin_amdgcn_readlane(rows, j);
        } else {
            r = rows;
            if (j + 1 < a.k) rows = a.rows[(size_t)t * a.k + j + 1];
        }
        if ((unsigned)r >= (unsigned)a.R || c >= a.K) continue;
        *reinterpret_cast<u32x2 *>(a.codes + (size_t)r * a.K + c) = code;
        if ((lane & 15) == 0) a.scales[(size_t)block * a.R + r] = scale;
    }
}

// A wave: four rows of four blocks.
template <int DT>
__global__ void __launch_bounds__(256)
dequantize_rows_kernel(const uint8_t *__restrict__ codes, const float *__restrict__ scales, uint16_t *__restrict__ x, int R, int K) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const long long r = ((long long)blockIdx.z * gridDim.x + blockIdx.x) * kDequantRows + wid * 4 + (lane >> 4);
    if (r >= R) return;
    const int block0 = blockIdx.y * kQuantBlocks, c0 = block0 * 128 + (lane & 15) * 8;
    u32x2 c[kQuantBlocks];
    float s[kQuantBlocks];
#pragma unroll
    for (int p = 0; p < kQuantBlocks; ++p) {
        const int at = c0 + p * 128;
        c[p] = u32x2{0u, 0u};
        s[p] = 0.0f;
        if (at < K) {
            c[p] = *reinterpret_cast<const u32x2 *>(codes + (size_t)r * K + at);
            s[p] = scales[(size_t)(block0 + p) * R + r];
        }
    }
#pragma unroll
    for (int p = 0; p < kQuantBlocks; ++p) {
        const int at = c0 + p * 128;
        if (at < K) __builtin_nontemporal_store(from_f8<DT>(c[p], s[p]), reinterpret_cast<u32x4 *>(x + (size_t)r * K + at));
    }
}

// Grid: groups of `per` rows along x and, beyond 2^20 of them, z; groups of blocks along y.
inline dim3 quant_grid(int rows, int K, int per, int blocks) {
    const int groups = ceil_div(rows, per), z = ceil_div(groups, 1 << 20);
    return dim3((unsigned)ceil_div(groups, z), (unsigned)ceil_div(ceil_div(K, 128), blocks), (unsigned)z);
}

// ------------------------------------------------------------------ weights --

struct QuantWeights {
    const uint16_t *w;        // [E][N][K]
    uint8_t *codes, *codes_t; // [E][N][K] and [E][K][N], either null
    float *scales, *scales_t; // [E][N blocks][K blocks] and [E][K blocks][N blocks]
    int E, N, K;
    int pow2;
};

// A workgroup takes one block of 128 x 128: a thread 16 bytes of 8 of its rows. The transposed codes go through
// LDS as bytes: rows of 128 + 4 (columns of 4 codes then leave in other banks).
template <int DT>
__global__ void __launch_bounds__(256)
quantize_weights_kernel(QuantWeights a) {
    __shared__ uint32_t top_smem[4];
    __shared__ __attribute__((aligned(16))) uint8_t tile[128 * 132];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int nb = ceil_div(a.N, 128), kb = ceil_div(a.K, 128);
    const long long block = (long long)blockIdx.y * gridDim.x + blockIdx.x;
    if (block >= (long long)a.E * nb * kb) return;
    const int number = (int)block, k = number % kb, n = number / kb % nb, e = number / kb / nb;
    const int col = k * 128 + (tid & 15) * 8;
    u32x4 v[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // (The first value in the place of one outside: with a branch for each load the compiler made one array of 32
        // registers of these, copied for each, and 234 registers in all: twice the time.)
        const int row = n * 128 + i * 16 + (tid >> 4);
        const bool there = row < a.N && col < a.K;
        const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(a.w + (there ? ((size_t)e * a.N + row) * a.K + col : 0)));
        v[i] = there ? x : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, top_bits(v[i]));
#pragma unroll
    for (int s = 1; s < 64; s *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, s));
    if (lane == 0) top_smem[wid] = top;
    __syncthreads();
    top = max(max(top_smem[0], top_smem[1]), max(top_smem[2], top_smem[3]));
    float scale, by;
    block_scale(to_f32<DT>(top), a.pow2 != 0, scale, by);
    if (tid == 0) {
        if (a.scales) a.scales[((size_t)e * nb + n) * kb + k] = scale;
        if (a.scales_t) a.scales_t[((size_t)e * kb + k) * nb + n] = scale;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 16 + (tid >> 4), row = n * 128 + r;
        const u32x2 c = to_f8<DT>(v[i], by);
        if (a.codes && row < a.N && col < a.K) *reinterpret_cast<u32x2 *>(a.codes + ((size_t)e * a.N + row) * a.K + col) = c;
        if (a.codes_t) {
            uint32_t *const at = reinterpret_cast<uint32_t *>(tile + r * 132 + (tid & 15) * 8);
            at[0] = c.x;
            at[1] = c.y;
        }
    }
    if (!a.codes_t) return;
    __syncthreads();
    // Thread: 16 codes along N of 4 columns of K, whose words of 4 x 4 codes turn in registers.
    const int r0 = (tid & 7) * 16, q0 = tid >> 3;
    u32x4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = reinterpret_cast<const uint32_t *>(tile)[(r0 + 4 * i + j) * 33 + q0];
        const uint32_t a0 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), a1 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
        const uint32_t b0 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), b1 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
        o[0][i] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
        o[1][i] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
        o[2][i] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
        o[3][i] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = k * 128 + 4 * q0 + i;
        if (c < a.K && n * 128 + r0 < a.N)   // N is a multiple of 16
            *reinterpret_cast<u32x4 *>(a.codes_t + ((size_t)e * a.K + c) * a.N + n * 128 + r0) = o[i];
    }
}

// x [E][N][K] from codes and scales [E][N blocks][K blocks]. A wave takes eight rows of four blocks of one expert: a row's 1 KiB
// leave together.
constexpr int kDequantWeightRows = 32;   // of a workgroup: within one block of 128

template <int DT>
__global__ void __launch_bounds__(256)
dequantize_weights_kernel(const uint8_t *__restrict__ codes, const float *__restrict__ scales, uint16_t *__restrict__ x, int E, int N, int K) {
    constexpr int R = kDequantWeightRows / 4;
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int nb = ceil_div(N, 128), kb = ceil_div(K, 128), parts = ceil_div(N, kDequantWeightRows), wide = ceil_div(kb, kQuantBlocks);
    const long long unit = (long long)blockIdx.y * gridDim.x + blockIdx.x;
    if (unit >= (long long)E * parts * wide) return;
    const int number = (int)unit, n0 = number / wide % parts * kDequantWeightRows + wid * R, e = number / wide / parts;
    const int k = number % wide * kQuantBlocks + (lane >> 4), col = k * 128 + (lane & 15) * 8;
    if (col >= K) return;
    const float s = scales[((size_t)e * nb + n0 / 128) * kb + k];
    u32x2 c[R];
#pragma unroll
    for (int i = 0; i < R; ++i)   // (the last row in the place of one past it)
        c[i] = *reinterpret_cast<const u32x2 *>(codes + ((size_t)e * N + min(n0 + i, N - 1)) * K + col);
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (n0 + i < N) __builtin_nontemporal_store(from_f8<DT>(c[i], s), reinterpret_cast<u32x4 *>(x + ((size_t)e * N + n0 + i) * K + col));
}

}  // namespace gbm
