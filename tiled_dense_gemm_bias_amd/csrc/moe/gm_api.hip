// C ABI of libgba_moe (declared in gba_moe.h): argument checks, device check, choice of kernel, launch.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "../experts/gx_reduce.hpp"
#include "gba_moe.h"
#include "gm_fp8.hpp"
#include "gm_launch.hpp"
#include "gm_move.hpp"
#include "gm_plan.hpp"
#include "gm_route.hpp"

#define GBM_VERSION_STRING "0.1.0"

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

bool is16(int dtype) { return dtype == GBA_DTYPE_F16 || dtype == GBA_DTYPE_BF16; }

size_t size3(int64_t a, int64_t b, int64_t c) { return (size_t)a * (size_t)b * (size_t)c; }

// Rows and slots are 32-bit numbers; a row's length leaves room for a tile's 32-bit byte offsets.
constexpr int64_t kMaxRows = 1LL << 29, kMaxWidth = 1LL << 23, kMaxDepth = 1LL << 22;

bool bad_sort(int64_t T, int64_t E, int64_t k) {
    return T < 0 || E < 1 || E > gbm::kMaxExperts || k < 1 || k > gbm::kMaxTop || T > kMaxRows / k;
}
bool bad_route(int64_t T, int64_t E, int64_t k) { return bad_sort(T, E, k) || k > E; }

// ------------------------------------------------------------------- sorting --

// Slots that one workgroup sorts, beyond which each block of a larger grid counts its own first; blocks of such a grid
// (each adds up all blocks' counts).
constexpr int kBlockSlots = 2048, kMaxBlocks = 256;

// Tokens a block: as few as 256 blocks leave, in whole sixteens (four waves of a routing block with up to 256 experts;
// a wave's pass takes some 10 us whatever the others do, so that few tokens belong on many CUs).
constexpr int kLeastTokens = 16;

void sort_shape(int64_t T, int64_t E, int64_t k, int *tokens, int *blocks) {
    int64_t per = (T + kMaxBlocks - 1) / kMaxBlocks;
    per = T * k <= kBlockSlots ? T : (per + kLeastTokens - 1) / kLeastTokens * kLeastTokens;
    if (per < 1) per = 1;
    *tokens = (int)per;
    *blocks = T ? (int)((T + per - 1) / per) : 1;
}

size_t sort_bytes(int64_t T, int64_t E, int64_t k) {
    int tokens, blocks;
    sort_shape(T, E, k, &tokens, &blocks);
    return blocks > 1 ? size3(blocks, gbm::count_pitch((int)E), 4) : 0;
}

gbm::Sort sort_of(const int32_t *indices, const void *counts, int32_t *offsets, int32_t *rows, int32_t *slots, int64_t T, int64_t E,
                  int64_t k) {
    int tokens, blocks;
    sort_shape(T, E, k, &tokens, &blocks);
    return {indices, (const int32_t *)counts, offsets, rows, slots, (int)(T * k), (int)E, (int)(tokens * k), blocks};
}

hipError_t launch_sort(const gbm::Sort &s) {
    return gbm::launch(s.E <= 256 ? gbm::sort_kernel<256> : gbm::sort_kernel<1024>, dim3(s.blocks), dim3(gbm::kRouteThreads), t_stream, s);
}

template <bool GROUPED>
hipError_t launch_route(const gbm::Route &a, const gbm::Sort &s, int64_t blocks) {
    const int waves = (a.tokens * (a.E <= 256 ? 16 : a.E <= 512 ? 32 : 64) + 63) / 64;   // of one pass
    const dim3 grid = gba::tile_grid(blocks);
    const dim3 block(s.indices || waves > gbm::kRouteWaves ? gbm::kRouteThreads : waves * 64);
    void (*kernel)(gbm::Route, gbm::Sort) = a.E <= 16    ? gbm::route_kernel<16, 1, GROUPED>
                                            : a.E <= 32  ? gbm::route_kernel<16, 2, GROUPED>
                                            : a.E <= 64  ? gbm::route_kernel<16, 4, GROUPED>
                                            : a.E <= 128 ? gbm::route_kernel<16, 8, GROUPED>
                                            : a.E <= 256 ? gbm::route_kernel<16, 16, GROUPED>
                                            : a.E <= 512 ? gbm::route_kernel<32, 16, GROUPED>
                                                         : gbm::route_kernel<64, 16, GROUPED>;
    return gbm::launch(kernel, grid, block, t_stream, a, s);
}

// ------------------------------------------------------------------- products --

int check_product(int64_t T, int64_t E, int64_t N, int64_t K) {
    if (T < 0 || N < 0 || K < 0 || E < 1 || E > GBM_MAX_GROUPS || T > kMaxRows || N > kMaxWidth || K > kMaxDepth) return GBA_ERR_SHAPE;
    return (K % 16) || (N % 8) ? GBA_ERR_ALIGN : GBA_OK;
}

int f8_product(const void *a_codes, const float *a_scales, const int32_t *offsets, bool grouped, const void *w_codes,
               const float *w_scales, const void *bias, const void *z, void *C, void *preact, int64_t T, int64_t E, int64_t N, int64_t K,
               int act, int dtype, bool slope, void *workspace, size_t workspace_bytes) {
    if (!is16(dtype)) return GBA_ERR_DTYPE;
    if (act < GBA_ACT_NONE || act > GBA_ACT_GELU_TANH) return GBA_ERR_ACT;
    int s = check_product(T, E, N, K);
    if (s) return s;
    const int64_t kb = (K + 127) / 128, nb = (N + 127) / 128;
    const Span spans[] = {{a_codes, size3(T, K, 1), true, false, 16},
                          {a_scales, size3(T, kb, 4), true, false, 4},
                          {offsets, (size_t)(E + 1) * 4, grouped && T > 0 && N > 0, false, 4},
                          {w_codes, size3(E, N, K), T > 0, false, 16},
                          {w_scales, size3(E * nb, kb, 4), T > 0, false, 4},
                          {bias, size3(E, N, 2), false, false, 16},
                          {z, size3(T, N, 2), slope && act != GBA_ACT_NONE, false, 16},
                          {C, size3(T, N, 2), true, true, 16},
                          {preact, size3(T, N, 2), false, true, 16},
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
    g.z = (const uint16_t *)z;
    g.C = C;
    g.zout = (uint16_t *)preact;
    g.T = (int)T;
    g.E = (int)E;
    g.N = (int)N;
    g.K = (int)(K / 2);   // 16-bit words of two codes
    g.act = act;
    g.splits = 1;
    int cus;
    if ((s = hip_result(gba::current_cus(&cus)))) return s;
    const gbm::Plan p = gbm::plan_f8(T, E, N, K, workspace ? workspace_bytes : 0, cus);
    if (p.kind == GBM_STREAM) return hip_result((slope ? gbm::f8_stream_slope : gbm::f8_stream_act)[dtype](g, t_stream));
    if (p.kind == GBM_PERSISTENT) {
        const gbx::LaunchFn *const big[2][2] = {{gbm::big_f8_act_f16, gbm::big_f8_act_bf16}, {gbm::big_f8_slope_f16, gbm::big_f8_slope_bf16}};
        return hip_result(big[slope][dtype][act](g, t_stream));
    }
    if (p.splits == 1) return hip_result((slope ? gbm::f8_slope : gbm::f8_act)[dtype][p.tile](g, t_stream));
    g.splits = p.splits;
    g.part = (float *)workspace;
    if ((s = hip_result(gbm::f8_part[p.tile](g, t_stream)))) return s;
    const gbx::LaunchFn reduce[2][2] = {{gbx::launch_reduce<gbx::EPI_ACT, 0, false>, gbx::launch_reduce<gbx::EPI_ACT, 1, false>},
                                        {gbx::launch_reduce<gbx::EPI_SLOPE, 0, false>, gbx::launch_reduce<gbx::EPI_SLOPE, 1, false>}};
    return hip_result(reduce[slope][dtype](g, t_stream));
}

}  // namespace

extern "C" {

const char *gbm_version(void) { return GBM_VERSION_STRING; }
int gbm_last_hip_error(void) { return t_last_hip; }
int gbm_set_stream(void *s) {
    t_stream = (hipStream_t)s;
    return GBA_OK;
}

size_t moe_sort_workspace(int64_t T, int64_t E, int64_t k) { return bad_sort(T, E, k) ? 0 : sort_bytes(T, E, k); }

int moe_route(const void *logits, const float *bias, int32_t *indices, float *weights, int32_t *offsets, int32_t *rows, int32_t *slots,
              int64_t T, int64_t E, int64_t k, int64_t groups, int64_t top_groups, int group_best, int score, float scale, int dtype,
              int flags, void *workspace, size_t workspace_bytes) {
    if (!is16(dtype) && dtype != GBM_DTYPE_F32) return GBA_ERR_DTYPE;
    if (score != GBM_SOFTMAX && score != GBM_SIGMOID) return GBA_ERR_ACT;
    if (flags & ~GBM_RENORMALIZE) return GBA_ERR_SHAPE;
    if (bad_route(T, E, k) || !isfinite(scale)) return GBA_ERR_SHAPE;
    if (groups < 1 || groups > gbm::kMaxGroups || E % groups || top_groups < 1 || top_groups > groups || group_best < 1 ||
        group_best > 2 || k > E / groups * top_groups)
        return GBA_ERR_SHAPE;
    const bool sort = offsets || rows || slots;
    const unsigned size = dtype == GBM_DTYPE_F32 ? 4 : 2;
    const Span spans[] = {{logits, size3(T, E, size), true, false, size},
                          {bias, size3(E, 4, 1), false, false, 4},
                          {indices, size3(T, k, 4), true, true, 4},
                          {weights, size3(T, k, 4), true, true, 4},
                          {offsets, size3(E + 1, 4, 1), sort, true, 4},
                          {rows, size3(T, k, 4), sort, true, 4},
                          {slots, size3(T, k, 4), false, true, 4},
                          {workspace, workspace_bytes, false, true, 16}};
    int s = check_spans(spans);
    if (s) return s;
    if (sort && workspace_bytes < sort_bytes(T, E, k)) return GBA_ERR_SCRATCH;
    if (sort && sort_bytes(T, E, k) && !workspace) return GBA_ERR_NULL;
    if (T == 0 && !sort) return GBA_OK;
    if ((s = check_device())) return s;
    gbm::Sort order = sort_of(indices, workspace, offsets, rows, slots, T, E, k);
    if (T > 0) {
        const bool counted = sort && order.blocks > 1;
        gbm::Route a = {};
        a.x = logits;
        a.bias = bias;
        a.indices = indices;
        a.weights = weights;
        a.counts = counted ? (int32_t *)workspace : nullptr;
        a.T = (int)T;
        a.E = (int)E;
        a.k = (int)k;
        a.groups = (int)groups;
        a.top_groups = (int)top_groups;
        a.group_best = group_best;
        a.group_size = (int)(E / groups);
        a.score = score;
        a.renorm = (flags & GBM_RENORMALIZE) != 0;
        a.dtype = dtype;
        a.scale = scale;
        // One block that sorts as well, where its waves are few enough. One block and two kernels, us: up to 16 tokens 4.2 to 10.5 and
        // 5.5 to 11.6 for any E (256 grouped experts 10.5, 11.6). 32 tokens: 32 experts 5.2, 6.3; 64 5.8, 6.7; 128 7.1, 7.5 (16
        // slots each 7.9, 8.3; grouped 9.5, 9.4), but 160 10.5, 9.8; 256 10.2, 9.4; grouped 13.2, 12.0. 64 tokens: 16 experts 5.3, 6.1;
        // 32 6.1, 6.4 (16 slots 8.3, 7.5), but 64 7.2, 6.7; 128 9.5, 7.5.
        const bool fused = sort && !counted && E <= 256 && T <= (E <= 32 ? gbm::kRouteWaves * 4 : E <= 128 ? 32 : 16);
        a.tokens = fused ? (int)T : counted ? order.per_block / (int)k : kLeastTokens;
        // Grouped keys fill a CU's LDS for 16 waves, however many work: as many as there are tokens for (16384 x 256 31 us with four).
        if (groups > top_groups && E > 64 && !fused && !counted)
            a.tokens = (int)std::min<int64_t>(((T + kMaxBlocks - 1) / kMaxBlocks + kLeastTokens - 1) / kLeastTokens * kLeastTokens, 64);
        gbm::Sort inside = order;
        if (!fused) inside.indices = nullptr;
        const int64_t n = (T + a.tokens - 1) / a.tokens;
        if ((s = hip_result(groups > top_groups ? launch_route<true>(a, inside, n) : launch_route<false>(a, inside, n))) || fused) return s;
    }
    return sort ? hip_result(launch_sort(order)) : GBA_OK;
}

int moe_route_grad(const void *logits, const int32_t *indices, const float *dweights, void *dlogits, int64_t T, int64_t E, int64_t k,
                   int score, float scale, int dtype, int flags) {
    if (!is16(dtype) && dtype != GBM_DTYPE_F32) return GBA_ERR_DTYPE;
    if (score != GBM_SOFTMAX && score != GBM_SIGMOID) return GBA_ERR_ACT;
    if (flags & ~GBM_RENORMALIZE) return GBA_ERR_SHAPE;
    if (bad_route(T, E, k) || !isfinite(scale)) return GBA_ERR_SHAPE;
    const unsigned size = dtype == GBM_DTYPE_F32 ? 4 : 2;
    const Span spans[] = {{logits, size3(T, E, size), true, false, size},
                          {indices, size3(T, k, 4), true, false, 4},
                          {dweights, size3(T, k, 4), true, false, 4},
                          {dlogits, size3(T, E, size), true, true, size}};
    int s = check_spans(spans);
    if (s) return s;
    if (T == 0) return GBA_OK;
    if ((s = check_device())) return s;
    gbm::RouteGrad a = {logits, indices, dweights, dlogits, (int)T, (int)E, (int)k, score, (flags & GBM_RENORMALIZE) != 0, dtype, scale};
    void (*kernel)(gbm::RouteGrad) = E <= 16    ? gbm::route_grad_kernel<16, 1>
                                     : E <= 32  ? gbm::route_grad_kernel<16, 2>
                                     : E <= 64  ? gbm::route_grad_kernel<16, 4>
                                     : E <= 128 ? gbm::route_grad_kernel<16, 8>
                                     : E <= 256 ? gbm::route_grad_kernel<16, 16>
                                     : E <= 512 ? gbm::route_grad_kernel<64, 8>
                                                : gbm::route_grad_kernel<64, 16>;
    const int64_t rows = gbm::kGradWaves * (E <= 256 ? 4 : 1);
    return hip_result(gbm::launch(kernel, gba::tile_grid((T + rows - 1) / rows), dim3(gbm::kGradWaves * 64), t_stream, a));
}

int moe_sort(const int32_t *indices, int32_t *offsets, int32_t *rows, int32_t *slots, int64_t T, int64_t E, int64_t k, void *workspace,
             size_t workspace_bytes) {
    if (bad_sort(T, E, k)) return GBA_ERR_SHAPE;
    const Span spans[] = {{indices, size3(T, k, 4), true, false, 4},
                          {offsets, size3(E + 1, 4, 1), true, true, 4},
                          {rows, size3(T, k, 4), true, true, 4},
                          {slots, size3(T, k, 4), false, true, 4},
                          {workspace, workspace_bytes, false, true, 16}};
    int s = check_spans(spans);
    if (s) return s;
    if (workspace_bytes < sort_bytes(T, E, k)) return GBA_ERR_SCRATCH;
    if (sort_bytes(T, E, k) && !workspace) return GBA_ERR_NULL;
    if ((s = check_device())) return s;
    const gbm::Sort order = sort_of(indices, workspace, offsets, rows, slots, T, E, k);
    if (order.blocks > 1) {
        s = hip_result(gbm::launch(gbm::count_kernel, dim3(order.blocks), dim3(gbm::kRouteThreads), t_stream, indices, (int32_t *)workspace,
                                   order.n, order.E, order.per_block));
        if (s) return s;
    }
    return hip_result(launch_sort(order));
}

// combine's dtype: the experts' rows', and whether the tokens' are in 32 bits.
static bool split_dtype(int dtype, int *rows, bool *f32) {
    *rows = dtype & ~GBM_F32_TOKENS;
    *f32 = (dtype & GBM_F32_TOKENS) != 0;
    return is16(*rows);
}

// Tokens, slots, columns and experts' rows of the moves.
static int check_move(int64_t T, int64_t k, int64_t H, int64_t R) {
    if (T < 0 || k < 1 || k > gbm::kMaxTop || H < 0 || R < 0 || T > kMaxRows / k || R > kMaxRows || H > kMaxWidth) return GBA_ERR_SHAPE;
    return H % 8 ? GBA_ERR_ALIGN : GBA_OK;
}

int moe_dispatch(const void *x, const int32_t *rows, void *out, int64_t T, int64_t k, int64_t H, int64_t R, int dtype) {
    if (!is16(dtype)) return GBA_ERR_DTYPE;
    int s = check_move(T, k, H, R);
    if (s) return s;
    const Span spans[] = {{x, size3(T, H, 2), true, false, 16},
                          {rows, size3(T, k, 4), H > 0, false, 4},
                          {out, size3(R, H, 2), true, true, 16}};
    if ((s = check_spans(spans))) return s;
    if (T == 0 || H == 0 || R == 0) return GBA_OK;
    if ((s = check_device())) return s;
    gbm::Move a = {};
    a.x = x;
    a.rows = rows;
    a.out = out;
    a.T = (int)T;
    a.k = (int)k;
    a.H = (int)H;
    a.R = (int)R;
    const int pieces = gba::ceil_div((int)H, gbm::kMoveThreads * 8);
    return hip_result(gbm::launch(gbm::dispatch_kernel, gbm::move_grid(T, pieces), dim3(gbm::kMoveThreads), t_stream, a));
}

int moe_combine(const void *y, const int32_t *rows, const float *weights, void *out, int64_t T, int64_t k, int64_t H, int64_t R,
                int dtype) {
    int dt;
    bool f32;
    if (!split_dtype(dtype, &dt, &f32)) return GBA_ERR_DTYPE;
    int s = check_move(T, k, H, R);
    if (s) return s;
    const Span spans[] = {{y, size3(R, H, 2), true, false, 16},
                          {rows, size3(T, k, 4), H > 0, false, 4},
                          {weights, size3(T, k, 4), false, false, 4},
                          {out, size3(T, H, f32 ? 4 : 2), true, true, 16}};
    if ((s = check_spans(spans))) return s;
    if (T == 0 || H == 0) return GBA_OK;
    if ((s = check_device())) return s;
    gbm::Move a = {};
    a.y = (const uint16_t *)y;
    a.rows = rows;
    a.w = weights;
    a.out = out;
    a.T = (int)T;
    a.k = (int)k;
    a.H = (int)H;
    a.R = (int)R;
    const int pieces = gba::ceil_div((int)H, gbm::kMoveThreads * 8);
    void (*const kernels[2][2])(gbm::Move) = {{gbm::combine_kernel<0, false>, gbm::combine_kernel<0, true>},
                                              {gbm::combine_kernel<1, false>, gbm::combine_kernel<1, true>}};
    return hip_result(gbm::launch(kernels[dt][f32], gbm::move_grid(T, pieces), dim3(gbm::kMoveThreads), t_stream, a));
}

int moe_combine_grad(const void *dout, const void *y, const int32_t *rows, const float *weights, void *dy, float *dweights, int64_t T,
                     int64_t k, int64_t H, int64_t R, int dtype) {
    int dt;
    bool f32;
    if (!split_dtype(dtype, &dt, &f32)) return GBA_ERR_DTYPE;
    int s = check_move(T, k, H, R);
    if (s) return s;
    const Span spans[] = {{dout, size3(T, H, f32 ? 4 : 2), true, false, 16},
                          {y, size3(R, H, 2), true, false, 16},
                          {rows, size3(T, k, 4), true, false, 4},
                          {weights, size3(T, k, 4), false, false, 4},
                          {dy, size3(R, H, 2), false, true, 16},
                          {dweights, size3(T, k, 4), false, true, 4}};
    if ((s = check_spans(spans))) return s;
    if (T == 0 || (!dy && !dweights)) return GBA_OK;
    if ((s = check_device())) return s;
    gbm::Move a = {};
    a.x = dout;
    a.y = (const uint16_t *)y;
    a.rows = rows;
    a.w = weights;
    a.dy = (uint16_t *)dy;
    a.dw = dweights;
    a.T = (int)T;
    a.k = (int)k;
    a.H = (int)H;
    a.R = (int)R;
    const bool one = gbm::one_wave_a_token(T, (int)H);
    void (*const kernels[2][2][2])(gbm::Move) = {
        {{gbm::combine_grad_kernel<0, 4, false>, gbm::combine_grad_kernel<0, 4, true>}, {gbm::combine_grad_kernel<0, 1, false>, gbm::combine_grad_kernel<0, 1, true>}},
        {{gbm::combine_grad_kernel<1, 4, false>, gbm::combine_grad_kernel<1, 4, true>}, {gbm::combine_grad_kernel<1, 1, false>, gbm::combine_grad_kernel<1, 1, true>}}};
    return hip_result(gbm::launch(kernels[dt][one][f32], gbm::move_grid(one ? (T + 3) / 4 : T, 1), dim3(gbm::kMoveThreads), t_stream, a));
}

int fp8_quantize(const void *X, const int32_t *rows, void *codes, float *scales, int64_t T, int64_t k, int64_t K, int64_t R, int dtype,
                 int flags) {
    if (!is16(dtype)) return GBA_ERR_DTYPE;
    if (flags & ~GBM_POW2_SCALES) return GBA_ERR_SHAPE;
    if (T < 0 || k < 1 || k > gbm::kMaxTop || K < 0 || R < 0 || T > kMaxRows / k || R > kMaxRows || K > kMaxWidth) return GBA_ERR_SHAPE;
    if (!rows && (k != 1 || R != T)) return GBA_ERR_SHAPE;
    if (K % 16) return GBA_ERR_ALIGN;
    const Span spans[] = {{X, size3(T, K, 2), true, false, 16},
                          {rows, size3(T, k, 4), false, false, 4},
                          {codes, size3(R, K, 1), true, true, 16},
                          {scales, size3(R, (K + 127) / 128, 4), true, true, 4}};
    int s = check_spans(spans);
    if (s) return s;
    if (T == 0 || K == 0 || R == 0) return GBA_OK;
    if ((s = check_device())) return s;
    gbm::QuantRows a = {(const uint16_t *)X, rows, (uint8_t *)codes, scales, (int)T, (int)K, (int)k, (int)R, (flags & GBM_POW2_SCALES) != 0};
    void (*const kernels[2][3])(gbm::QuantRows) = {{gbm::quantize_rows_kernel<0, 1>, gbm::quantize_rows_kernel<0, 2>, gbm::quantize_rows_kernel<0, 4>},
                                                   {gbm::quantize_rows_kernel<1, 1>, gbm::quantize_rows_kernel<1, 2>, gbm::quantize_rows_kernel<1, 4>}};
    const int which = K <= 128 ? 0 : K <= 256 ? 1 : 2, blocks = 1 << which;
    return hip_result(gbm::launch(kernels[dtype][which], gbm::quant_grid((int)T, (int)K, 4 * gbm::kQuantBlocks / blocks, blocks), dim3(256),
                                  t_stream, a));
}

int fp8_dequantize(const void *codes, const float *scales, void *X, int64_t R, int64_t K, int dtype) {
    if (!is16(dtype)) return GBA_ERR_DTYPE;
    if (R < 0 || K < 0 || R > kMaxRows || K > kMaxWidth) return GBA_ERR_SHAPE;
    if (K % 16) return GBA_ERR_ALIGN;
    const Span spans[] = {{X, size3(R, K, 2), true, true, 16},
                          {codes, size3(R, K, 1), true, false, 16},
                          {scales, size3(R, (K + 127) / 128, 4), true, false, 4}};
    int s = check_spans(spans);
    if (s) return s;
    if (R == 0 || K == 0) return GBA_OK;
    if ((s = check_device())) return s;
    auto *const kernel = dtype == GBA_DTYPE_F16 ? gbm::dequantize_rows_kernel<0> : gbm::dequantize_rows_kernel<1>;
    return hip_result(gbm::launch(kernel, gbm::quant_grid((int)R, (int)K, gbm::kDequantRows, gbm::kQuantBlocks), dim3(256), t_stream, (const uint8_t *)codes, scales,
                                  (uint16_t *)X, (int)R, (int)K));
}

int fp8_quantize_weights(const void *W, void *codes, float *scales, void *codes_t, float *scales_t, int64_t E, int64_t N, int64_t K,
                         int dtype, int flags) {
    if (!is16(dtype)) return GBA_ERR_DTYPE;
    if (flags & ~GBM_POW2_SCALES) return GBA_ERR_SHAPE;
    if (E < 0 || N < 0 || K < 0 || E > GBM_MAX_GROUPS || N > kMaxWidth || K > kMaxWidth) return GBA_ERR_SHAPE;
    if ((K % 16) || (codes_t && N % 16)) return GBA_ERR_ALIGN;
    if (!codes != !scales || !codes_t != !scales_t) return GBA_ERR_NULL;
    const int64_t nb = (N + 127) / 128, kb = (K + 127) / 128;
    if (E * nb > 0x3fffffffLL / (kb ? kb : 1)) return GBA_ERR_SHAPE;
    const Span spans[] = {{W, size3(E, N * 2, K), true, false, 16},
                          {codes, size3(E, N, K), codes_t == nullptr, true, 16},
                          {scales, size3(E * nb, kb, 4), codes_t == nullptr, true, 4},
                          {codes_t, size3(E, N, K), false, true, 16},
                          {scales_t, size3(E * nb, kb, 4), false, true, 4}};
    int s = check_spans(spans);
    if (s) return s;
    if (E == 0 || N == 0 || K == 0) return GBA_OK;
    if ((s = check_device())) return s;
    gbm::QuantWeights a = {(const uint16_t *)W, (uint8_t *)codes, (uint8_t *)codes_t, scales, scales_t, (int)E, (int)N, (int)K,
                           (flags & GBM_POW2_SCALES) != 0};
    auto *const kernel = dtype == GBA_DTYPE_F16 ? gbm::quantize_weights_kernel<0> : gbm::quantize_weights_kernel<1>;
    return hip_result(gbm::launch(kernel, gba::tile_grid(E * nb * kb), dim3(256), t_stream, a));
}

int fp8_dequantize_weights(const void *codes, const float *scales, void *W, int64_t E, int64_t N, int64_t K, int dtype) {
    if (!is16(dtype)) return GBA_ERR_DTYPE;
    if (E < 0 || N < 0 || K < 0 || E > GBM_MAX_GROUPS || N > kMaxWidth || K > kMaxWidth) return GBA_ERR_SHAPE;
    if (K % 16) return GBA_ERR_ALIGN;
    const int64_t nb = (N + 127) / 128, kb = (K + 127) / 128;
    if (E * nb > 0x3fffffffLL / (kb ? kb : 1)) return GBA_ERR_SHAPE;
    const Span spans[] = {{W, size3(E, N * 2, K), true, true, 16},
                          {codes, size3(E, N, K), true, false, 16},
                          {scales, size3(E * nb, kb, 4), true, false, 4}};
    int s = check_spans(spans);
    if (s) return s;
    if (E == 0 || N == 0 || K == 0) return GBA_OK;
    if ((s = check_device())) return s;
    auto *const kernel = dtype == GBA_DTYPE_F16 ? gbm::dequantize_weights_kernel<0> : gbm::dequantize_weights_kernel<1>;
    const int64_t units = E * ((N + gbm::kDequantWeightRows - 1) / gbm::kDequantWeightRows) * ((kb + gbm::kQuantBlocks - 1) / gbm::kQuantBlocks);
    return hip_result(gbm::launch(kernel, gba::tile_grid(units), dim3(256), t_stream, (const uint8_t *)codes, scales, (uint16_t *)W, (int)E,
                                  (int)N, (int)K));
}

int gemm_bias_act_fp8_block(const void *a_codes, const float *a_scales, const void *w_codes, const float *w_scales, const void *bias,
                            void *C, void *preact, int64_t M, int64_t N, int64_t K, int act, int dtype, void *workspace,
                            size_t workspace_bytes) {
    return f8_product(a_codes, a_scales, nullptr, false, w_codes, w_scales, bias, nullptr, C, preact, M, 1, N, K, act, dtype, false,
                      workspace, workspace_bytes);
}

int grouped_gemm_bias_act_fp8_block(const void *a_codes, const float *a_scales, const int32_t *offsets, const void *w_codes,
                                    const float *w_scales, const void *bias, void *C, void *preact, int64_t T, int64_t E, int64_t N,
                                    int64_t K, int act, int dtype, void *workspace, size_t workspace_bytes) {
    return f8_product(a_codes, a_scales, offsets, true, w_codes, w_scales, bias, nullptr, C, preact, T, E, N, K, act, dtype, false,
                      workspace, workspace_bytes);
}

int gemm_act_grad_fp8_block(const void *dc_codes, const float *dc_scales, const void *w_codes, const float *w_scales, const void *z,
                            void *dA, int64_t M, int64_t N, int64_t K, int act, int dtype, void *workspace, size_t workspace_bytes) {
    return f8_product(dc_codes, dc_scales, nullptr, false, w_codes, w_scales, nullptr, z, dA, nullptr, M, 1, N, K, act, dtype, true,
                      workspace, workspace_bytes);
}

int grouped_gemm_act_grad_fp8_block(const void *dc_codes, const float *dc_scales, const int32_t *offsets, const void *w_codes,
                                    const float *w_scales, const void *z, void *dA, int64_t T, int64_t E, int64_t N, int64_t K, int act,
                                    int dtype, void *workspace, size_t workspace_bytes) {
    return f8_product(dc_codes, dc_scales, offsets, true, w_codes, w_scales, nullptr, z, dA, nullptr, T, E, N, K, act, dtype, true,
                      workspace, workspace_bytes);
}

int gbm_get_plan(int64_t T, int64_t E, int64_t N, int64_t K, size_t workspace_bytes, int cus, gbm_plan *plan) {
    if (!plan) return GBA_ERR_NULL;
    const int s = check_product(T, E, N, K);
    if (s) return s;
    if (T < 1 || N < 1 || K < 1 || cus < 1) return GBA_ERR_SHAPE;
    const gbm::Plan p = gbm::plan_f8(T, E, N, K, workspace_bytes, cus);
    const gbx::TileCost &t = p.kind == GBM_PERSISTENT ? gbm::kBig : p.kind == GBM_STREAM ? gbm::kStream : gbm::kRowTiles[p.tile];
    *plan = {p.kind, (int32_t)t.bm, (int32_t)t.bn, p.splits};
    return GBA_OK;
}

}  // extern "C"
