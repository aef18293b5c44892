// What the kernels of libgba_experts share: the groups (gx_groups.hpp), activation slopes,
// the epilogue of eight outputs, and the microscaled 4-bit matrix instruction.
#pragma once

#include "gba_dma.hpp"
#include "gemm_v3.hpp"   // mfma16x16x32, aswz, bswz
#include "gx_groups.hpp"

namespace gbx {

using namespace gba;

// Launches a kernel and returns that launch's status. (hipGetLastError after a launch would also
// report what an earlier call of this thread left, and a split product stop half way.)
template <class T>
struct Exactly {
    using type = T;
};
template <class... Args>
hipError_t launch(void (*kernel)(Args...), dim3 grid, dim3 block, hipStream_t stream, typename Exactly<Args>::type... args) {
    void *pointers[] = {&args...};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, block, pointers, 0, stream);
}

// Operand types. MX4 rows are counted in 16-bit words of four codes: a row of K
// values is K / 4 words, and a 64-word slice (128 bytes) is 256 values, so the
// 4-bit kernels move the same bytes in the same tiles as the 16-bit ones; only
// the matrix instruction and its scales differ. F8 rows (8-bit floats with fp32 scales by blocks of 128)
// are K / 2 words, a slice 128 values: one block, and one matrix instruction of 128.
enum { OP_F16 = 0, OP_BF16 = 1, OP_MX4 = 2, OP_F8 = 3 };

// What the kernel does with a tile's fp32 sums.
enum {
    EPI_ACT = 0,    // act(sum + bias), and the rounded sum + bias where asked for
    EPI_SLOPE = 1,  // sum * act'(z)
    EPI_GRAD = 2,   // the sum, rounded or fp32, or added to what is there
    EPI_PART = 3    // fp32 partial sums of one split
};

// expert_rows for a uniform e, into scalar registers by scalar loads (no kernel
// writes the offsets), which wait for no vector memory.
__device__ __forceinline__ void expert_rows_uniform(const Group &g, int e, int &start, int &rows) {
    int lo = 0, hi = g.T;
    if (g.offsets) {
        typedef const int32_t __attribute__((address_space(4))) *ScalarPtr;
        const ScalarPtr o = (ScalarPtr)(uintptr_t)g.offsets;
        lo = o[e];
        hi = o[e + 1];
    }
    rows_between(lo, hi, g.T, start, rows);
    start = __builtin_amdgcn_readfirstlane(start);
    rows = __builtin_amdgcn_readfirstlane(rows);
}

// ------------------------------------------------------- activation slopes --

// act'(z) in fp32. relu'(0) = 0; at z = +-inf the limit; NaN for NaN.
//  sigmoid:   t / (1 + t)^2 with t = e^-|z| (no cancellation on either side).
//  softplus:  the logistic of z.
//  gelu:      Phi(z) + z phi(z) = q for z <= 0 and 1 - q for z > 0, with x = |z|,
//             q = e^(-x^2/2) (R(t) - x / sqrt(2 pi)), t = 1 / (1 + x/4): R, of degree 7,
//             is fitted to m(x) / sqrt(2 pi), m the Mills ratio Phi(-x) / phi(x), for q's
//             relative error (tiled_dense_gemm_bias_amd/gelu_slope_fit.py): within 2e-7,
//             and for z < -1 within (1 + z^2/8) 3e-7 of itself (the rounding of the
//             exponential's argument; z^2 is exact, as z has 16 bits). x is clamped
//             outside the exponential only: at z = +-inf q is 0 and NaN stays NaN.
//  gelu_tanh: z = tanh form; with s = 1 / (1 + e), e = e^(-2y),
//             y = sqrt(2/pi) (z + c z^3): s + z s (1 - s) 2 y', and 1 - s = e s.
//             Outside |z| = 10 the slope is 0 or 1 to 1e-30: z is clamped there,
//             which keeps e finite.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    constexpr float kLog2e = 1.4426950408889634f;
    if constexpr (ACT == ACT_RELU) {
        return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    } else if constexpr (ACT == ACT_SIGMOID) {
        const float t = __builtin_amdgcn_exp2f(-fabsf(z) * kLog2e);
        const float r = __builtin_amdgcn_rcpf(1.0f + t);
        return t * r * r;
    } else if constexpr (ACT == ACT_SOFTPLUS) {
        return act_fn<ACT_SIGMOID>(z);
    } else if constexpr (ACT == ACT_GELU) {
        const float a = fminf(fabsf(z), 16.0f);
        const float t = __builtin_amdgcn_rcpf(fmaf(a, 0.25f, 1.0f));
        // R and x / sqrt(2 pi) by 1/8, the exponential by 8: the hardware's exponential is 0
        // below 2^-126, and q, which is up to 5 times that there, would be lost sooner.
        constexpr float s = 0.125f;
        float r = fmaf(t, s * -0.0971691083497504f, s * 0.3682747148994894f);
        r = fmaf(t, r, s * -0.3203441591740204f);
        r = fmaf(t, r, s * 0.3387267891725851f);
        r = fmaf(t, r, s * -0.0111699049002808f);
        r = fmaf(t, r, s * 0.1251299008583134f);
        r = fmaf(t, r, s * 0.0963644464504781f);
        r = fmaf(t, r, s * 0.0001873002465777f);
        const float p = fmaf(a, s * -0.3989422804014327f, r);
        const float q = p * __builtin_amdgcn_exp2f(fmaf(z * z, -0.5f * kLog2e, 3.0f));
        return z > 0.0f ? 1.0f - q : q;
    } else if constexpr (ACT == ACT_GELU_TANH) {
        const float c = fminf(fmaxf(z, -10.0f), 10.0f);
        const float c2 = c * c;
        const float e = __builtin_amdgcn_exp2f(-c * fmaf(c2, 0.10294324159622192f, 2.302208185195923f));
        const float s = __builtin_amdgcn_rcpf(1.0f + e);
        // 2 y' = 2 sqrt(2/pi) (1 + 3 c z^2) = 1.5957691 + 0.21406545 z^2
        const float r = fmaf(c * (e * s) * s, fmaf(c2, 0.21406544f, 1.5957691216057308f), s);
        return z != z ? z : r;
    } else {
        return 1.0f;
    }
}

// f(std::integral_constant<int, act>{}) for the run-time act (uniform).
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>{}); break;
    case ACT_SIGMOID: f(std::integral_constant<int, ACT_SIGMOID>{}); break;
    case ACT_GELU: f(std::integral_constant<int, ACT_GELU>{}); break;
    case ACT_SOFTPLUS: f(std::integral_constant<int, ACT_SOFTPLUS>{}); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, ACT_NONE>{}); break;
    }
}

// ----------------------------------------------------- eight outputs at once --

template <int DT>
__device__ __forceinline__ void load8(const uint16_t *p, f32x4 (&v)[2]) {
    const u32x4 x = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i / 2][2 * (i % 2)] = to_f32<DT>(x[i] & 0xffffu);
        v[i / 2][2 * (i % 2) + 1] = to_f32<DT>(x[i] >> 16);
    }
}

template <int DT>
__device__ __forceinline__ void store8(uint16_t *p, const f32x4 (&v)[2]) {
    const u32x4 x = {pack2<DT>(v[0][0], v[0][1]), pack2<DT>(v[0][2], v[0][3]),
                     pack2<DT>(v[1][0], v[1][1]), pack2<DT>(v[1][2], v[1][3])};
    __builtin_nontemporal_store(x, reinterpret_cast<u32x4 *>(p));
}

// The epilogue of eight adjacent sums of one row of expert e, from column n on,
// at place `at` of the output.
template <int EPI, int ODT>
__device__ __forceinline__ void finish(const Group &g, f32x4 (&v)[2], int e, int n, size_t at) {
    if constexpr (EPI == EPI_ACT) {
        if (g.bias) {
            f32x4 bias[2];
            load8<ODT>(g.bias + (size_t)e * g.N + n, bias);
            v[0] += bias[0];
            v[1] += bias[1];
        }
        if (g.zout) store8<ODT>(g.zout + at, v);
        with_act(g.act, [&](auto act_c) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i / 4][i % 4] = act_fn<decltype(act_c)::value>(v[i / 4][i % 4]);
        });
        store8<ODT>((uint16_t *)g.C + at, v);
    } else if constexpr (EPI == EPI_SLOPE) {
        if (g.act != ACT_NONE) {
            f32x4 z[2];
            load8<ODT>(g.z + at, z);
            with_act(g.act, [&](auto act_c) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i / 4][i % 4] *= act_slope<decltype(act_c)::value>(z[i / 4][i % 4]);
            });
        }
        store8<ODT>((uint16_t *)g.C + at, v);
    } else if (g.flags & GF_F32) {
        f32x4 *const p = reinterpret_cast<f32x4 *>((float *)g.C + at);
        const bool add = (g.flags & GF_ADD) != 0;
        p[0] = add ? p[0] + v[0] : v[0];
        p[1] = add ? p[1] + v[1] : v[1];
    } else {
        store8<ODT>((uint16_t *)g.C + at, v);
    }
}

// ------------------------------------------------------------------- MX4 ----

typedef int i32x8 __attribute__((ext_vector_type(8)));

// c + A.B on 16 x 16 x 128 blocks of 4-bit codes: lane l holds row / column l % 16
// and the 32 codes of block l / 16 (16 bytes), and in the low byte of its scale
// operand that block's exponent. Results lie as those of the 16-bit 16x16x32 instruction.
__device__ __forceinline__ f32x4 mfma_mx4(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
    const i32x8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// A.B on 16 x 16 x 128 blocks of 8-bit codes (E4M3): lane l holds row / column l % 16 and 32 codes, the same
// places of the 128 in both operands. Results lie as those of the 16-bit 16x16x32 instruction.
__device__ __forceinline__ f32x4 mfma_f8(const i32x8 &a, const i32x8 &b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

}  // namespace gbx
