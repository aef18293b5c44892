// What the kernels of libgba_experts share: the arguments of a grouped product,
// the search for the expert and tile of a work unit, activation slopes, and the
// microscaled 4-bit matrix instruction.
#pragma once

#include "gba_dma.hpp"
#include "gemm_v3.hpp"   // mfma16x16x32, aswz, bswz

namespace gbx {

using namespace gba;

// Operand types. MX4 rows are counted in 16-bit words of four codes: a row of K
// values is K / 4 words, and a 64-word slice (128 bytes) is 256 values, so the
// 4-bit kernels move the same bytes in the same tiles as the 16-bit ones; only
// the matrix instruction and its scales differ.
enum { OP_F16 = 0, OP_BF16 = 1, OP_MX4 = 2 };

// What the kernel does with a tile's fp32 sums.
enum {
    EPI_ACT = 0,    // act(sum + bias), and the rounded sum + bias where asked for
    EPI_SLOPE = 1,  // sum * act'(z)
    EPI_GRAD = 2,   // the sum, rounded or fp32, or added to what is there
    EPI_PART = 3    // fp32 partial sums of one split
};

// A grouped product. Rows mode (weight gradients: see wgrad below): the rows of expert e of A [T][K] times
// B_e, giving rows of C [T][N]. wgrad: At_e^T.B_e over the rows of expert e, with
// At [T][M] and B [T][N], giving C [E][M][N]. K counts 16-bit words.
struct Group {
    const uint16_t *A, *B;
    const uint32_t *sa, *sb;     // MX4 scale planes of A and B, one dword a row
    const int32_t *offsets;      // null: one expert, all T rows
    const uint16_t *bias;        // [E][N] or null
    const uint16_t *z;           // EPI_SLOPE: [T][N]
    void *C;
    uint16_t *zout;              // EPI_ACT: [T][N] or null
    void *sums;                  // EPI_GRAD: [E][columns of dC] or null
    float *part;                 // EPI_PART: [splits][rows of C][N]
    int T, E, M, N, K;
    int act, flags, splits;
    int row_bound;               // rows mode: most row tiles the grid was made for
};
// EPI_GRAD: fp32 output, added to what is there; B read once and too large to stay in the caches.
enum { GF_F32 = 1, GF_ADD = 2, GF_STREAM = 4 };

__device__ __forceinline__ int clamp_row(int v, int T) { return min(max(v, 0), T); }

// First row and row count of expert e: offsets clamped to [0, T].
__device__ __forceinline__ void expert_rows(const Group &g, int e, int &start, int &rows) {
    if (!g.offsets) {
        start = 0;
        rows = g.T;
        return;
    }
    start = clamp_row(g.offsets[e], g.T);
    rows = max(clamp_row(g.offsets[e + 1], g.T) - start, 0);
}

// The same for a uniform e, into scalar registers by scalar loads (no kernel
// writes the offsets), which wait for no vector memory.
__device__ __forceinline__ void expert_rows_uniform(const Group &g, int e, int &start, int &rows) {
    int lo = 0, hi = g.T;
    if (g.offsets) {
        typedef const int32_t __attribute__((address_space(4))) *ScalarPtr;
        const ScalarPtr o = (ScalarPtr)(uintptr_t)g.offsets;
        lo = o[e];
        hi = o[e + 1];
    }
    start = __builtin_amdgcn_readfirstlane(clamp_row(lo, g.T));
    rows = __builtin_amdgcn_readfirstlane(max(clamp_row(hi, g.T) - start, 0));
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Row tiles of all experts (rows mode), each wave for itself: lane l takes
// experts l, l + 64, ... Offsets that decrease can name more tiles than the
// grid was made for; those are left out.
__device__ __forceinline__ int total_row_tiles(const Group &g, int bm, int lane) {
    long long n = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        int t = 0;
        if (e0 + lane < g.E) {
            int start, rows;
            expert_rows(g, e0 + lane, start, rows);
            t = ceil_div(rows, bm);
        }
        n += t;
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) n += __shfl_xor(n, d);
    return __builtin_amdgcn_readfirstlane((int)min(n, (long long)g.row_bound));
}

// Most row tiles that T rows of E experts can make: one for each full tile, and
// one more for each expert that has rows.
inline long long row_tile_bound(long long T, long long E, int bm) {
    return T / bm + (E < T ? E : T);
}

// The expert that row tile number t (in expert order) lies in, with the number of
// row tiles before it, its tiles, rows and first row; `total` is that of total_row_tiles, and the
// rest is set where t < total. Every lane gets the same answer.
struct Found {
    int e, before, tiles, start, rows, total;
};
__device__ __forceinline__ Found found_at(int e0, unsigned long long past, int before, int upto, int n, int start, int rows) {
    const int l = __builtin_amdgcn_readfirstlane(__ffsll(past) - 1);
    Found f;
    f.e = e0 + l;
    f.tiles = __builtin_amdgcn_readlane(n, l);
    f.before = before + __builtin_amdgcn_readlane(upto, l) - f.tiles;
    f.start = __builtin_amdgcn_readlane(start, l);
    f.rows = __builtin_amdgcn_readlane(rows, l);
    return f;
}
__device__ __forceinline__ Found find_row_tile(const Group &g, int bm, int t, int lane) {
    Found f = {0, 0, 0, 0, 0, 0};
    int before = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        int n = 0, start = 0, rows = 0;
        if (e0 + lane < g.E) {
            expert_rows(g, e0 + lane, start, rows);
            n = ceil_div(rows, bm);
        }
        const int upto = wave_scan(n, lane);
        const unsigned long long past = __ballot(before + upto > t);
        if (past) {
            f = found_at(e0, past, before, upto, n, start, rows);
            break;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return f;
}

// For up to 64 experts, one reading of the offsets for both the total and the
// tile: `tile_of(total)` gives the row tile wanted, or -1.
template <class F>
__device__ __forceinline__ Found locate_few(const Group &g, int bm, int lane, F &&tile_of) {
    int n = 0, start = 0, rows = 0;
    if (lane < g.E) {
        expert_rows(g, lane, start, rows);
        n = ceil_div(rows, bm);
    }
    const int upto = wave_scan(n, lane);
    const int total = min(__builtin_amdgcn_readlane(upto, 63), g.row_bound);
    const int t = tile_of(total);
    Found f = {0, 0, 0, 0, 0, total};
    const unsigned long long past = __ballot(upto > t);
    if (t >= 0 && past) {
        f = found_at(0, past, 0, upto, n, start, rows);
        f.total = total;
    }
    return f;
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

}  // namespace gbx
