/* Host-side check program for the AddressSanitizer / UndefinedBehaviorSanitizer build of
 * libgba_moe's host code (tests/test_host_sanitizers_moe_cpu.py builds and runs it):
 * argument errors of every entry point, sizes and addresses at their limits, and the choice of
 * kernel over drawn sizes. No call here reaches a launch: each fails a host-side check, has nothing to
 * do, or finds no device; as a second guard the program runs only where no GPU is
 * visible (exit 77 otherwise). Prints "host sanitize check ok" and exits 0 when every check holds. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gba_moe.h"

/* HIP runtime (C linkage; 0 is hipSuccess). */
extern int hipGetDeviceCount(int *count);

static int g_fail = 0;
#define CHECK(cond)                                                             \
    do {                                                                        \
        if (!(cond)) {                                                          \
            fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
            g_fail = 1;                                                         \
        }                                                                       \
    } while (0)

/* Aligned addresses far apart, never followed. */
static void *at(int i) { return (void *)(((uintptr_t)i << 48) + 0x10000); }
static const int64_t kBad[] = {-1, INT64_MIN, INT64_MAX, (int64_t)1 << 31, (int64_t)1 << 62};
enum { BAD = sizeof kBad / sizeof *kBad };

/* One call of each entry point with sizes d = {T, E or H, k or K, R or N} and one output. */
enum { ROUTE, ROUTE_GRAD, SORT, DISPATCH, COMBINE, COMBINE_GRAD, QUANT, DEQUANT, QUANT_W, DEQUANT_W, FWD, GROUPED_FWD, GRAD, GROUPED_GRAD, OPS };
static int call(int op, const int64_t *d, void *out, int dtype, int flags, void *ws, size_t nb) {
    switch (op) {
    case ROUTE:
        return moe_route(at(1), at(2), out, at(4), at(5), at(6), at(7), d[0], d[1], d[2], 1, 1, 1, 0, 1.0f, dtype, flags, ws, nb);
    case ROUTE_GRAD:
        return moe_route_grad(at(1), at(2), at(3), out, d[0], d[1], d[2], 0, 1.0f, dtype, flags);
    case SORT:
        return moe_sort(at(1), at(2), out, at(4), d[0], d[1], d[2], ws, nb);
    case DISPATCH:
        return moe_dispatch(at(1), at(2), out, d[0], d[2], d[1], d[3], dtype);
    case COMBINE:
        return moe_combine(at(1), at(2), at(3), out, d[0], d[2], d[1], d[3], dtype);
    case COMBINE_GRAD:
        return moe_combine_grad(at(1), at(2), at(3), at(4), out, at(6), d[0], d[2], d[1], d[3], dtype);
    case QUANT:
        return fp8_quantize(at(1), at(2), out, at(4), d[0], d[2], d[1], d[3], dtype, flags);
    case DEQUANT:
        return fp8_dequantize(at(1), at(2), out, d[3], d[1], dtype);
    case QUANT_W:
        return fp8_quantize_weights(at(1), out, at(3), at(4), at(5), d[0], d[3], d[1], dtype, flags);
    case DEQUANT_W:
        return fp8_dequantize_weights(at(1), at(2), out, d[0], d[3], d[1], dtype);
    case FWD:
        return gemm_bias_act_fp8_block(at(1), at(2), at(3), at(4), at(5), out, at(7), d[0], d[3], d[1], 3, dtype, ws, nb);
    case GROUPED_FWD:
        return grouped_gemm_bias_act_fp8_block(at(1), at(2), at(3), at(4), at(5), at(6), out, at(8), d[0], d[2], d[3], d[1], 3, dtype, ws, nb);
    case GRAD:
        return gemm_act_grad_fp8_block(at(1), at(2), at(3), at(4), at(5), out, d[0], d[3], d[1], 3, dtype, ws, nb);
    default:
        return grouped_gemm_act_grad_fp8_block(at(1), at(2), at(3), at(4), at(5), at(6), out, d[0], d[2], d[3], d[1], 3, dtype, ws, nb);
    }
}

static void argument_errors(void) {
    for (int op = 0; op < OPS; ++op) {
        const int64_t d[4] = {64, 64, op == QUANT ? 1 : 2, 64};
        const int typed = op != SORT, product = op >= FWD;
        const int uses[4] = {op != DEQUANT, 1, op < FWD ? op < DEQUANT : op == GROUPED_FWD || op == GROUPED_GRAD, op > SORT};
        CHECK(call(op, d, at(9), 0, 0, NULL, 0) == GBA_ERR_DEVICE);
        if (typed) CHECK(call(op, d, at(9), 7, 0, NULL, 0) == GBA_ERR_DTYPE);
        if (op <= ROUTE_GRAD || op == QUANT || op == QUANT_W) CHECK(call(op, d, at(9), 0, 1 << 30, NULL, 0) == GBA_ERR_SHAPE);
        if (op != COMBINE_GRAD) CHECK(call(op, d, NULL, 0, 0, NULL, 0) == GBA_ERR_NULL);
        CHECK(call(op, d, (char *)at(9) + 1, 0, 0, NULL, 0) == GBA_ERR_ALIGN);
        CHECK(call(op, d, at(1), 0, 0, NULL, 0) == GBA_ERR_ALIAS);
        CHECK(call(op, d, (void *)(UINTPTR_MAX - 15), 0, 0, NULL, 0) == GBA_ERR_DEVICE);
        if (op == ROUTE || op == SORT || product) {
            CHECK(call(op, d, at(9), 0, 0, at(1), SIZE_MAX) == GBA_ERR_ALIAS);
            CHECK(call(op, d, at(9), 0, 0, (void *)16, SIZE_MAX) == GBA_ERR_ALIAS);
            CHECK(call(op, d, at(9), 0, 0, (char *)at(20) + 8, 64) == GBA_ERR_ALIGN);
        }
        for (int w = 0; w < 4; ++w)
            for (int i = 0; i < BAD; ++i) {
                int64_t v[4] = {d[0], d[1], d[2], d[3]};
                v[w] = kBad[i];
                if (uses[w]) CHECK(call(op, v, at(9), 0, 0, NULL, 0) == GBA_ERR_SHAPE);
            }
    }
    /* The largest sizes, whose products come near 2^62 bytes: refused for what overlaps. */
    const int64_t rows = (int64_t)1 << 29, wide = (int64_t)1 << 23, deep = (int64_t)1 << 22;
    CHECK(moe_dispatch(at(1), at(2), at(1), rows / 2, 2, wide, rows, 0) == GBA_ERR_ALIAS);
    CHECK(fp8_quantize(at(1), at(2), at(1), at(3), rows / 32, 32, wide, rows, 0, 0) == GBA_ERR_ALIAS);
    CHECK(grouped_gemm_bias_act_fp8_block(at(1), at(2), at(3), at(4), at(5), at(6), at(1), NULL, rows, 4096, wide, deep, 0, 0, NULL, 0) == GBA_ERR_ALIAS);
    CHECK(fp8_quantize_weights(at(1), at(1), at(2), NULL, NULL, 1, wide, 16384 * 128 - 128, 0, 0) == GBA_ERR_ALIAS);
    CHECK(fp8_quantize_weights(at(1), at(2), at(3), NULL, NULL, 4096, wide, wide, 0, 0) == GBA_ERR_SHAPE);
    CHECK(moe_route(at(1), NULL, at(1), at(4), NULL, NULL, NULL, rows / 32, 1024, 32, 1, 1, 1, 0, 1.0f, 2, 0, NULL, 0) == GBA_ERR_ALIAS);
    /* Routing's own. */
#define ROUTED(G, TOP, BEST, SCORE, SCALE, WS, NB) \
    moe_route(at(1), at(2), at(3), at(4), at(5), at(6), at(7), 4096, 64, 8, G, TOP, BEST, SCORE, SCALE, 2, 0, WS, NB)
    const size_t nb = moe_sort_workspace(4096, 64, 8);
    CHECK(nb > 0 && ROUTED(8, 4, 2, 1, 1.0f, at(9), nb) == GBA_ERR_DEVICE);
    CHECK(ROUTED(8, 4, 2, 1, 1.0f, at(9), nb - 1) == GBA_ERR_SCRATCH && ROUTED(8, 4, 2, 1, 1.0f, NULL, nb) == GBA_ERR_NULL);
    for (int i = 0; i < BAD; ++i) {
        CHECK(ROUTED(kBad[i], 4, 2, 1, 1.0f, at(9), nb) == GBA_ERR_SHAPE);
        CHECK(ROUTED(8, kBad[i], 2, 1, 1.0f, at(9), nb) == GBA_ERR_SHAPE);
        CHECK(ROUTED(8, 4, (int)kBad[i], 1, 1.0f, at(9), nb) == GBA_ERR_SHAPE);
        CHECK(moe_sort_workspace(kBad[i], 64, 8) == 0 && moe_sort_workspace(64, kBad[i], 8) == 0 && moe_sort_workspace(64, 64, kBad[i]) == 0);
    }
    CHECK(ROUTED(8, 4, 2, 2, 1.0f, at(9), nb) == GBA_ERR_ACT && ROUTED(8, 4, 2, -1, 1.0f, at(9), nb) == GBA_ERR_ACT);
    CHECK(ROUTED(8, 4, 2, 1, INFINITY, at(9), nb) == GBA_ERR_SHAPE && ROUTED(8, 4, 2, 1, NAN, at(9), nb) == GBA_ERR_SHAPE);
    CHECK(moe_route(at(1), NULL, at(3), at(4), NULL, NULL, NULL, 0, 64, 8, 1, 1, 1, 0, 1.0f, 2, 0, NULL, 0) == GBA_OK);
}

static uint64_t g_state = 88172645463325252ull;
static uint64_t rnd(void) {   /* xorshift (Marsaglia, 2003) */
    g_state ^= g_state << 13;
    g_state ^= g_state >> 7;
    g_state ^= g_state << 17;
    return g_state;
}
/* Evenly over the logarithm of [1, 2^bits]. */
static int64_t spread(int bits) {
    const int b = (int)(rnd() % (uint64_t)(bits + 1));
    return ((int64_t)1 << b) + (int64_t)(rnd() % ((uint64_t)1 << b)) * (b < bits);
}

static void plans(void) {
    gbm_plan p;
    for (int i = 0; i < 200000; ++i) {
        const int64_t T = spread(29), E = spread(12), N = spread(20) * 8, K = spread(18) * 16;
        const int cus = (int)spread(12);
        const size_t nb = (size_t)spread(62);
        memset(&p, 0xff, sizeof p);
        CHECK(gbm_get_plan(T, E, N, K, nb, cus, &p) == GBA_OK);
        CHECK(p.kind >= GBM_RING && p.kind <= GBM_STREAM && p.tile_m >= 16 && p.tile_m <= 256 && p.tile_n >= 16 && p.tile_n <= 256);
        CHECK(p.splits >= 1 && p.splits <= 16 && (p.splits == 1 || 4.0 * (double)p.splits * (double)T * (double)N <= (double)nb));
        CHECK(p.kind != GBM_PERSISTENT || K > 128);
    }
    CHECK(gbm_get_plan(1, 1, 8, 16, SIZE_MAX, INT32_MAX, &p) == GBA_OK);
    CHECK(gbm_get_plan(1, 1, 8, 16, 0, 1, NULL) == GBA_ERR_NULL);
    for (int i = 0; i < BAD; ++i) {
        CHECK(gbm_get_plan(kBad[i], 1, 8, 16, 0, 256, &p) == GBA_ERR_SHAPE);
        CHECK(gbm_get_plan(1, kBad[i], 8, 16, 0, 256, &p) == GBA_ERR_SHAPE);
        CHECK(gbm_get_plan(1, 1, kBad[i], 16, 0, 256, &p) == GBA_ERR_SHAPE);
        CHECK(gbm_get_plan(1, 1, 8, kBad[i], 0, 256, &p) == GBA_ERR_SHAPE);
    }
    /* Sorting's workspace over drawn sizes: at most 256 KiB per 256 experts. */
    for (int i = 0; i < 200000; ++i) {
        const int64_t E = spread(10), k = 1 + (int64_t)(rnd() % 32), T = spread(24);
        if (k <= E) CHECK(moe_sort_workspace(T, E, k) <= (size_t)((E + 255) / 256) * (256 << 10));
    }
}

int main(void) {
    int ndev = 0;
    if (hipGetDeviceCount(&ndev) == 0 && ndev > 0) {
        printf("a GPU is visible: this check runs only without one\n");
        return 77;
    }
    CHECK(strlen(gbm_version()) > 0 && gbm_set_stream(NULL) == GBA_OK);
    argument_errors();
    plans();
    if (g_fail) {
        fprintf(stderr, "host sanitize check: FAILED\n");
        return 1;
    }
    printf("host sanitize check ok\n");
    return 0;
}
