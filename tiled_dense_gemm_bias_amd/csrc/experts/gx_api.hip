// C ABI of libgba_experts (declared in gba_experts.h): argument checks, device
// check, choice of kernel, launch.
#include <string.h>

#include <mutex>

#include "gba_experts.h"
#include "gx_colsum.hpp"
#include "gx_launch.hpp"
#include "gx_mx4.hpp"
#include "gx_plan.hpp"
#include "gx_reduce.hpp"

#define GBX_VERSION_STRING "0.1.0"

namespace {

thread_local hipStream_t t_stream = nullptr;
thread_local int t_last_hip = 0;

int hip_result(hipError_t e) {
    if (e == hipSuccess) return GBA_OK;
    t_last_hip = (int)e;
    return GBA_ERR_HIP;
}

// GBA_OK when the current device is a gfx950.
int check_device() {
    static std::mutex mu;
    static int state[64];   // 0: not looked at, 1: gfx950, 2: another
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || dev < 0 || dev >= 64) {
        (void)hipGetLastError();
        t_last_hip = (int)e;
        return GBA_ERR_DEVICE;
    }
    std::lock_guard<std::mutex> lk(mu);
    if (!state[dev]) {
        hipDeviceProp_t p;
        e = hipGetDeviceProperties(&p, dev);
        if (e != hipSuccess) {
            (void)hipGetLastError();
            t_last_hip = (int)e;
            return GBA_ERR_DEVICE;
        }
        state[dev] = strncmp(p.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    }
    return state[dev] == 1 ? GBA_OK : GBA_ERR_DEVICE;
}

// ------------------------------------------------------------ argument checks --

// An array argument: where it is, how long, how it must be aligned.
struct Span {
    const void *p;
    size_t bytes;
    bool required, output;
    unsigned align;
};

bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y ? y - x < a.bytes : x - y < b.bytes;   // sums of address and size could wrap round
}

template <int N>
int check_spans(const Span (&s)[N]) {
    for (const Span &a : s)
        if (a.required && a.bytes && !a.p) return GBA_ERR_NULL;
    for (const Span &a : s)
        if (a.p && ((uintptr_t)a.p & (a.align - 1))) return GBA_ERR_ALIGN;
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j)
            if (i != j && s[i].output && overlap(s[i], s[j])) return GBA_ERR_ALIAS;
    return GBA_OK;
}

int check_enums(int act, int dtype) {
    if (dtype != GBA_DTYPE_F16 && dtype != GBA_DTYPE_BF16) return GBA_ERR_DTYPE;
    if (act < GBA_ACT_NONE || act > GBA_ACT_GELU_TANH) return GBA_ERR_ACT;
    return GBA_OK;
}

// Rows of a grouped product: 64 experts whose offsets decrease can claim 32 T rows
// between them, in tiles of 16, which stays a 32-bit count. Rows of a quantised matrix: a 32-bit index.
constexpr int64_t kMaxRows = 1LL << 29, kMaxQuantRows = 0x7fffffffLL;
// A row pitch inside a tile's 32-bit byte offsets: 256 K-contiguous rows, or 64 rows along K.
constexpr int64_t kMaxDepth = 1LL << 21, kMaxWidth = 1LL << 23;

int check_sizes(int64_t T, int64_t E, int64_t depth, int64_t width) {
    if (T < 0 || depth < 0 || width < 0 || E < 1 || E > GBX_MAX_EXPERTS) return GBA_ERR_SHAPE;
    if (T > kMaxRows || depth > kMaxDepth || width > kMaxWidth) return GBA_ERR_SHAPE;
    return GBA_OK;
}

size_t size3(int64_t a, int64_t b, int64_t c) { return (size_t)a * (size_t)b * (size_t)c; }

// The choice of kernel of every product, from the arguments of its call.
gbx::Plan plan_of(int op, int64_t T, int64_t E, int64_t N, int64_t K, size_t workspace, int cus) {
    switch (op) {
    case GBX_FORWARD: return gbx::plan_rows(T, E, N, K, workspace, cus);
    case GBX_ACT_GRAD: return gbx::plan_rows(T, E, K, N, workspace, cus);
    case GBX_MX4: return gbx::plan_rows(T, E, N, K / 4, workspace, cus);
    default: return gbx::plan_grad(T, E, K, N, op == GBX_WGRAD_BIAS, workspace, cus);
    }
}

// The ring kernel of a plan, then (a split) the second pass.
int launch_split(gbx::Group &g, const gbx::Plan &p, const gbx::LaunchFn &whole, const gbx::LaunchFn &part,
                 const gbx::LaunchFn &reduce, void *workspace) {
    if (p.stream) g.flags |= gbx::GF_STREAM;
    if (p.splits == 1) return hip_result(whole(g, t_stream));
    g.splits = p.splits;
    g.part = (float *)workspace;
    const int s = hip_result(part(g, t_stream));
    return s ? s : hip_result(reduce(g, t_stream));
}

int current_cus(int *cus) { return hip_result(gba::current_cus(cus)); }

}  // namespace

extern "C" {

const char *gbx_version(void) { return GBX_VERSION_STRING; }
int gbx_last_hip_error(void) { return t_last_hip; }
int gbx_set_stream(void *s) {
    t_stream = (hipStream_t)s;
    return GBA_OK;
}

int grouped_gemm_bias_act(const void *A, const int32_t *offsets, const void *W, const void *bias,
                          void *C, void *preact, int64_t T, int64_t E, int64_t N, int64_t K,
                          int act, int dtype, int flags, void *workspace, size_t workspace_bytes) {
    int s = check_enums(act, dtype);
    if (s) return s;
    if (flags & ~GBA_TRANSPOSE_B) return GBA_ERR_SHAPE;
    if ((s = check_sizes(T, E, K, N))) return s;
    if ((K % 8) || (N % 8)) return GBA_ERR_ALIGN;
    const Span spans[] = {{A, size3(T, K, 2), true, false, 16},
                          {offsets, (size_t)(E + 1) * 4, T > 0 && N > 0, false, 4},
                          {W, size3(E, N * 2, K), T > 0, false, 16},
                          {bias, size3(E, N, 2), false, false, 16},
                          {C, size3(T, N, 2), true, true, 16},
                          {preact, size3(T, N, 2), false, true, 16},
                          {workspace, workspace_bytes, false, true, 16}};
    if ((s = check_spans(spans))) return s;
    if (T == 0 || N == 0) return GBA_OK;
    if ((s = check_device())) return s;
    gbx::Group g = {};
    g.A = (const uint16_t *)A;
    g.B = (const uint16_t *)W;
    g.offsets = offsets;
    g.bias = (const uint16_t *)bias;
    g.C = C;
    g.zout = (uint16_t *)preact;
    g.T = (int)T;
    g.E = (int)E;
    g.N = (int)N;
    g.K = (int)K;
    g.act = act;
    g.splits = 1;
    const bool nt = (flags & GBA_TRANSPOSE_B) != 0;
    int cus;
    if ((s = current_cus(&cus))) return s;
    const gbx::Plan p = plan_of(GBX_FORWARD, T, E, N, K, workspace ? workspace_bytes : 0, cus);
    if (p.big) {
        const gbx::LaunchFn *const big[2][2] = {{gbx::big_fwd_nn_f16, gbx::big_fwd_nn_bf16},
                                                {gbx::big_fwd_nt_f16, gbx::big_fwd_nt_bf16}};
        return hip_result(big[nt][dtype][act](g, t_stream));
    }
    const gbx::LaunchFn reduce[2] = {gbx::launch_reduce<gbx::EPI_ACT, 0, false>, gbx::launch_reduce<gbx::EPI_ACT, 1, false>};
    return launch_split(g, p, (nt ? gbx::fwd_nt : gbx::fwd_nn)[dtype][p.tile],
                        (nt ? gbx::part_nt : gbx::part_nn)[dtype][p.tile], reduce[dtype], workspace);
}

int grouped_gemm_act_grad(const void *dC, const int32_t *offsets, const void *W, const void *z,
                          void *dA, int64_t T, int64_t E, int64_t N, int64_t K, int act, int dtype,
                          int flags, void *workspace, size_t workspace_bytes) {
    int s = check_enums(act, dtype);
    if (s) return s;
    if (flags & ~GBA_TRANSPOSE_B) return GBA_ERR_SHAPE;
    if ((s = check_sizes(T, E, N, K))) return s;
    if ((K % 8) || (N % 8)) return GBA_ERR_ALIGN;
    const Span spans[] = {{dC, size3(T, N, 2), true, false, 16},
                          {offsets, (size_t)(E + 1) * 4, T > 0 && K > 0, false, 4},
                          {W, size3(E, N * 2, K), T > 0, false, 16},
                          {z, size3(T, K, 2), act != GBA_ACT_NONE, false, 16},
                          {dA, size3(T, K, 2), true, true, 16},
                          {workspace, workspace_bytes, false, true, 16}};
    if ((s = check_spans(spans))) return s;
    if (T == 0 || K == 0) return GBA_OK;
    if ((s = check_device())) return s;
    gbx::Group g = {};
    g.A = (const uint16_t *)dC;
    g.B = (const uint16_t *)W;
    g.offsets = offsets;
    g.z = (const uint16_t *)z;
    g.C = dA;
    g.T = (int)T;
    g.E = (int)E;
    g.N = (int)K;   // the product's columns
    g.K = (int)N;   // and its depth
    g.act = act;
    g.splits = 1;
    // W [E,N,K] has its rows along the sum, W [E,K,N] its columns.
    const bool nt = !(flags & GBA_TRANSPOSE_B);
    int cus;
    if ((s = current_cus(&cus))) return s;
    const gbx::Plan p = plan_of(GBX_ACT_GRAD, T, E, N, K, workspace ? workspace_bytes : 0, cus);
    if (p.big) {
        const gbx::LaunchFn *const big[2][2] = {{gbx::big_slope_nn_f16, gbx::big_slope_nn_bf16},
                                                {gbx::big_slope_nt_f16, gbx::big_slope_nt_bf16}};
        return hip_result(big[nt][dtype][act](g, t_stream));
    }
    const gbx::LaunchFn reduce[2] = {gbx::launch_reduce<gbx::EPI_SLOPE, 0, false>, gbx::launch_reduce<gbx::EPI_SLOPE, 1, false>};
    return launch_split(g, p, (nt ? gbx::slope_nt : gbx::slope_nn)[dtype][p.tile],
                        (nt ? gbx::part_nt : gbx::part_nn)[dtype][p.tile], reduce[dtype], workspace);
}

int grouped_gemm_wgrad(const void *A, const void *dC, const int32_t *offsets, void *dW,
                       void *dbias, int64_t T, int64_t E, int64_t N, int64_t K, int dtype,
                       int flags, void *workspace, size_t workspace_bytes) {
    int s = check_enums(GBA_ACT_NONE, dtype);
    if (s) return s;
    if (flags & ~(GBA_TRANSPOSE_B | GBX_OUT_F32 | GBX_ACCUMULATE)) return GBA_ERR_SHAPE;
    if ((flags & GBX_ACCUMULATE) && !(flags & GBX_OUT_F32)) return GBA_ERR_DTYPE;
    if ((s = check_sizes(T, E, 0, N))) return s;
    if ((s = check_sizes(T, E, 0, K))) return s;
    if ((K % 8) || (N % 8)) return GBA_ERR_ALIGN;
    const size_t ob = (flags & GBX_OUT_F32) ? 4 : 2;
    const Span spans[] = {{A, size3(T, K, 2), true, false, 16},
                          {dC, size3(T, N, 2), true, false, 16},
                          {offsets, (size_t)(E + 1) * 4, N > 0, false, 4},
                          {dW, size3(E, N * ob, K), true, true, 16},
                          {dbias, size3(E, N, ob), false, true, 16},
                          {workspace, workspace_bytes, false, true, 16}};
    if ((s = check_spans(spans))) return s;
    if (N == 0) return GBA_OK;
    if ((s = check_device())) return s;
    const bool f32 = (flags & GBX_OUT_F32) != 0, add = (flags & GBX_ACCUMULATE) != 0;
    gbx::Group g = {};
    g.offsets = offsets;
    g.T = (int)T;
    g.E = (int)E;
    g.flags = (f32 ? gbx::GF_F32 : 0) | (add ? gbx::GF_ADD : 0);
    g.splits = 1;
    if (K > 0) {
        // Rows of the output: the columns of the first factor (dC with GBA_TRANSPOSE_B).
        const bool nk = (flags & GBA_TRANSPOSE_B) != 0;
        g.A = (const uint16_t *)(nk ? dC : A);
        g.B = (const uint16_t *)(nk ? A : dC);
        g.M = (int)(nk ? N : K);
        g.N = (int)(nk ? K : N);
        g.C = dW;
        int cus;
        if ((s = current_cus(&cus))) return s;
        const gbx::Plan p = plan_of(dbias ? GBX_WGRAD_BIAS : GBX_WGRAD, T, E, N, K, workspace ? workspace_bytes : 0, cus);
        const gbx::LaunchFn reduce[2] = {gbx::launch_reduce<gbx::EPI_GRAD, 0, true>, gbx::launch_reduce<gbx::EPI_GRAD, 1, true>};
        if (p.big) {   // with the bias gradient
            g.sums = dbias;
            const int kind = (f32 ? gbx::GRAD_F32 : gbx::GRAD_16) + (!dbias ? 0 : nk ? gbx::GRAD_SUMS_A : gbx::GRAD_SUMS_B);
            return hip_result(gbx::big_wgrad_tn[dtype][kind](g, t_stream));
        }
        s = launch_split(g, p, gbx::wgrad_tn[dtype][p.tile], gbx::part_tn[dtype][p.tile], reduce[dtype], workspace);
        if (s) return s;
    }
    if (dbias) {
        g.A = (const uint16_t *)dC;
        g.N = (int)N;
        g.C = dbias;
        return hip_result(gbx::launch_column_sums(g, dtype, t_stream));
    }
    return GBA_OK;
}

int mx4_quantize(const void *X, void *codes, void *scales, int64_t M, int64_t K, int dtype) {
    int s = check_enums(GBA_ACT_NONE, dtype);
    if (s) return s;
    if (M < 0 || K < 0 || M > kMaxQuantRows || K > kMaxWidth) return GBA_ERR_SHAPE;
    if (K % 32) return GBA_ERR_ALIGN;
    const Span spans[] = {{X, size3(M, K, 2), true, false, 16},
                          {codes, size3(M, K / 2, 1), true, true, 16},
                          {scales, size3(M, (K + 127) / 128, 4), true, true, 16}};
    if ((s = check_spans(spans))) return s;
    if (M == 0 || K == 0) return GBA_OK;
    if ((s = check_device())) return s;
    auto *const kernel = dtype == GBA_DTYPE_F16 ? gbx::mx4_quantize_kernel<0> : gbx::mx4_quantize_kernel<1>;
    return hip_result(gbx::launch(kernel, gbx::mx4_grid((int)M, (int)K), dim3(256), t_stream, (const uint16_t *)X,
                                  (uint32_t *)codes, (uint32_t *)scales, (int)M, (int)K));
}

int mx4_dequantize(const void *codes, const void *scales, void *X, int64_t M, int64_t K,
                   int dtype) {
    int s = check_enums(GBA_ACT_NONE, dtype);
    if (s) return s;
    if (M < 0 || K < 0 || M > kMaxQuantRows || K > kMaxWidth) return GBA_ERR_SHAPE;
    if (K % 32) return GBA_ERR_ALIGN;
    const Span spans[] = {{X, size3(M, K, 2), true, true, 16},
                          {codes, size3(M, K / 2, 1), true, false, 16},
                          {scales, size3(M, (K + 127) / 128, 4), true, false, 16}};
    if ((s = check_spans(spans))) return s;
    if (M == 0 || K == 0) return GBA_OK;
    if ((s = check_device())) return s;
    auto *const kernel = dtype == GBA_DTYPE_F16 ? gbx::mx4_dequantize_kernel<0> : gbx::mx4_dequantize_kernel<1>;
    return hip_result(gbx::launch(kernel, gbx::mx4_grid((int)M, (int)K), dim3(256), t_stream, (const uint32_t *)codes,
                                  (const uint32_t *)scales, (uint16_t *)X, (int)M, (int)K));
}

// offsets null: dense (E == 1).
static int mx4_common(const void *a_codes, const void *a_scales, const int32_t *offsets, bool grouped,
                      const void *w_codes, const void *w_scales, const void *bias, void *C,
                      int64_t T, int64_t E, int64_t N, int64_t K, int act, int dtype,
                      void *workspace, size_t workspace_bytes) {
    int s = check_enums(act, dtype);
    if (s) return s;
    if (K < 0 || K > 4 * kMaxDepth) return GBA_ERR_SHAPE;
    if ((s = check_sizes(T, E, 0, N))) return s;
    if ((K % 32) || (N % 8)) return GBA_ERR_ALIGN;
    const int64_t planes = (K + 127) / 128;
    const Span spans[] = {{a_codes, size3(T, K / 2, 1), true, false, 16},
                          {a_scales, size3(T, planes, 4), true, false, 16},
                          {offsets, (size_t)(E + 1) * 4, grouped && T > 0 && N > 0, false, 4},
                          {w_codes, size3(E, N, K / 2), T > 0, false, 16},
                          {w_scales, size3(E * N, planes, 4), T > 0, false, 16},
                          {bias, size3(E, N, 2), false, false, 16},
                          {C, size3(T, N, 2), true, true, 16},
                          {workspace, workspace_bytes, false, true, 16}};
    if ((s = check_spans(spans))) return s;
    if (T == 0 || N == 0) return GBA_OK;
    if ((s = check_device())) return s;
    gbx::Group g = {};
    g.A = (const uint16_t *)a_codes;
    g.B = (const uint16_t *)w_codes;
    g.sa = (const uint32_t *)a_scales;
    g.sb = (const uint32_t *)w_scales;
    g.offsets = grouped ? offsets : nullptr;
    g.bias = (const uint16_t *)bias;
    g.C = C;
    g.T = (int)T;
    g.E = (int)E;
    g.N = (int)N;
    g.K = (int)(K / 4);   // 16-bit words of four codes
    g.act = act;
    g.splits = 1;
    int cus;
    if ((s = current_cus(&cus))) return s;
    const gbx::Plan p = plan_of(GBX_MX4, T, E, N, K, workspace ? workspace_bytes : 0, cus);
    if (p.big)
        return hip_result((dtype == GBA_DTYPE_F16 ? gbx::big_mx4_f16 : gbx::big_mx4_bf16)[act](g, t_stream));
    const gbx::LaunchFn reduce[2] = {gbx::launch_reduce<gbx::EPI_ACT, 0, false>, gbx::launch_reduce<gbx::EPI_ACT, 1, false>};
    return launch_split(g, p, gbx::mx4_nt[dtype][p.tile], gbx::part_mx4[dtype][p.tile], reduce[dtype], workspace);
}

int gemm_bias_act_mx4(const void *a_codes, const void *a_scales, const void *w_codes,
                      const void *w_scales, const void *bias, void *C, int64_t M, int64_t N,
                      int64_t K, int act, int dtype, void *workspace, size_t workspace_bytes) {
    return mx4_common(a_codes, a_scales, nullptr, false, w_codes, w_scales, bias, C, M, 1, N, K, act, dtype,
                      workspace, workspace_bytes);
}

int gbx_get_plan(int op, int64_t T, int64_t E, int64_t N, int64_t K, size_t workspace_bytes,
                 int cus, gbx_plan *plan) {
    if (!plan) return GBA_ERR_NULL;
    if (op < GBX_FORWARD || op > GBX_MX4 || cus < 1 || T < 1 || N < 1 || K < 1) return GBA_ERR_SHAPE;
    const bool grad = op == GBX_WGRAD || op == GBX_WGRAD_BIAS;
    const int64_t depth = grad ? 0 : op == GBX_ACT_GRAD ? N : op == GBX_MX4 ? K / 4 : K;
    int s = check_sizes(T, E, depth, op == GBX_ACT_GRAD ? K : N);
    if (!s && grad) s = check_sizes(T, E, 0, K);
    if (s) return s;
    if ((K % (op == GBX_MX4 ? 32 : 8)) || (N % 8)) return GBA_ERR_ALIGN;
    const gbx::Plan p = plan_of(op, T, E, N, K, workspace_bytes, cus);
    const gbx::TileCost &t = p.big ? gbx::kBig : grad ? gbx::kGradTileCost[p.tile] : gbx::kRowTiles[p.tile];
    *plan = {t.bm, t.bn, p.big, p.splits, p.stream};
    return GBA_OK;
}

int grouped_gemm_bias_act_mx4(const void *a_codes, const void *a_scales, const int32_t *offsets,
                              const void *w_codes, const void *w_scales, const void *bias, void *C,
                              int64_t T, int64_t E, int64_t N, int64_t K, int act, int dtype,
                              void *workspace, size_t workspace_bytes) {
    return mx4_common(a_codes, a_scales, offsets, true, w_codes, w_scales, bias, C, T, E, N, K, act, dtype,
                      workspace, workspace_bytes);
}

}  // extern "C"
