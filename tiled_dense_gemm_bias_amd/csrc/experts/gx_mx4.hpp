// Microscaled 4-bit quantisation and its inverse. Both are bound by HBM: 2 bytes
// of one side and 17/32 of a byte of the other for each value (16384 x 8192 bf16: 70
// and 60 us, 4.9 and 5.7 TB/s; a large copy 5.0).
#pragma once

#include "gx_common.hpp"

namespace gbx {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// 2^(s - 127) for a scale byte s: 2^-127 is subnormal, 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23);
}

// The scale byte of a block whose largest magnitude has the bits `top` (the
// order of 16-bit float magnitudes is that of their bits): floor(log2) - 2 + 127,
// at least 0; 255 for infinities and NaN.
template <int DT>
__device__ __forceinline__ uint32_t block_scale(uint32_t top) {
    if constexpr (DT == DT_BF16) {
        const int e = (int)(top >> 7);
        return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
    } else {
        const int e = (int)(top >> 10);
        if (e == 31) return 255u;
        if (e > 0) return (uint32_t)(e - 15 - 2 + 127);
        return top == 0u ? 0u : (uint32_t)(31 - __clz((int)top) - 24 - 2 + 127);   // subnormal
    }
}

// Two values, as their bits, to two codes in byte SEL of `into`.
template <int DT, int SEL>
__device__ __forceinline__ uint32_t to_codes(uint32_t into, uint32_t two, float scale, bool tiny) {
    if constexpr (DT == DT_BF16) {
        // A scale of 2^-127 has no normal fp32 form: such values are scaled first
        // (exactly), then converted with scale 1.
        if (tiny)
            return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(into, to_f32<DT>(two & 0xffffu) * 0x1p127f,
                                                            to_f32<DT>(two >> 16) * 0x1p127f, 1.0f, SEL);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(into, __builtin_bit_cast(bf16x2_t, two), scale, SEL);
    } else {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(into, __builtin_bit_cast(f16x2_t, two), scale, SEL);
    }
}

// A wave takes 4 rows x 128 values, 16 lanes of 8 values a row; four lanes share
// a block. A workgroup's four waves are stacked along the rows, so that 16 rows'
// scale dwords of a plane are written side by side; it takes kQuantPlanes planes,
// whose loads all go out before the first is used (a wave has 4 KiB in flight).
constexpr int kQuantRows = 16, kQuantPlanes = 4;

template <int DT>
__global__ void __launch_bounds__(256)
mx4_quantize_kernel(const uint16_t *__restrict__ X, uint32_t *__restrict__ codes,
                    uint32_t *__restrict__ scales, int M, int K) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const long long row = ((long long)blockIdx.z * gridDim.x + blockIdx.x) * kQuantRows + wid * 4 + (lane >> 4);
    if (row >= M) return;   // whole 16-lane groups, so no block loses a lane
    const int plane0 = blockIdx.y * kQuantPlanes, k0 = plane0 * 128 + (lane & 15) * 8;
    const uint16_t *const x = X + (size_t)row * K;
    u32x4 v[kQuantPlanes];
#pragma unroll
    for (int p = 0; p < kQuantPlanes; ++p) {
        const int k = k0 + p * 128;
        v[p] = k < K ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x + k)) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int p = 0; p < kQuantPlanes; ++p) {
        const int k = k0 + p * 128;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t m = v[p][i] & 0x7fff7fffu;
            top = max(top, max(m & 0xffffu, m >> 16));
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const uint32_t s = block_scale<DT>(top);
        const float sc = scale_value(s == 255u ? 127u : s);
        const bool tiny = s == 0u;
        uint32_t c = 0;
        c = to_codes<DT, 0>(c, v[p][0], sc, tiny);
        c = to_codes<DT, 1>(c, v[p][1], sc, tiny);
        c = to_codes<DT, 2>(c, v[p][2], sc, tiny);
        c = to_codes<DT, 3>(c, v[p][3], sc, tiny);
        if (s == 255u) c = 0;
        if (k < K) codes[((size_t)row * K + k) >> 3] = c;
        // The four blocks' bytes, into the first lane of the row.
        uint32_t w = k < K ? s << (8 * ((lane >> 2) & 3)) : 0u;
        w |= (uint32_t)__shfl_xor((int)w, 4);
        w |= (uint32_t)__shfl_xor((int)w, 8);
        if ((lane & 15) == 0 && (plane0 + p) * 128 < K) scales[(size_t)(plane0 + p) * M + row] = w;
    }
}

template <int DT>
__global__ void __launch_bounds__(256)
mx4_dequantize_kernel(const uint32_t *__restrict__ codes, const uint32_t *__restrict__ scales,
                      uint16_t *__restrict__ X, int M, int K) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const long long row = ((long long)blockIdx.z * gridDim.x + blockIdx.x) * kQuantRows + wid * 4 + (lane >> 4);
    if (row >= M) return;
    const int plane0 = blockIdx.y * kQuantPlanes, k0 = plane0 * 128 + (lane & 15) * 8;
    uint32_t c[kQuantPlanes], w[kQuantPlanes];
#pragma unroll
    for (int p = 0; p < kQuantPlanes; ++p) {
        const int k = k0 + p * 128;
        c[p] = k < K ? codes[((size_t)row * K + k) >> 3] : 0u;
        w[p] = k < K ? scales[(size_t)(plane0 + p) * M + row] : 0u;
    }
#pragma unroll
    for (int p = 0; p < kQuantPlanes; ++p) {
        const int k = k0 + p * 128;
        const float sc = scale_value((w[p] >> (8 * ((lane >> 2) & 3))) & 255u);
        // The codes' values exactly, then one product (exact but for the ends of fp32's range).
        const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[p], 1.0f, 0);
        const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[p], 1.0f, 1);
        const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[p], 1.0f, 2);
        const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[p], 1.0f, 3);
        const u32x4 y = {pack2<DT>(v0[0] * sc, v0[1] * sc), pack2<DT>(v1[0] * sc, v1[1] * sc),
                         pack2<DT>(v2[0] * sc, v2[1] * sc), pack2<DT>(v3[0] * sc, v3[1] * sc)};
        if (k < K) __builtin_nontemporal_store(y, reinterpret_cast<u32x4 *>(X + (size_t)row * K + k));
    }
}

// Grid: 16-row groups along x and, beyond 2^20 of them, z; groups of planes along
// y (K <= 2^23: at most 2^14).
inline dim3 mx4_grid(int M, int K) {
    const int groups = ceil_div(M, kQuantRows), z = ceil_div(groups, 1 << 20);
    return dim3((unsigned)ceil_div(groups, z), (unsigned)ceil_div(ceil_div(K, 128), kQuantPlanes), (unsigned)z);
}

}  // namespace gbx
