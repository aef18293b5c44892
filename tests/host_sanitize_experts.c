/* Host-side check program for the AddressSanitizer / UndefinedBehaviorSanitizer build of
 * libgba_experts' host code (tests/test_host_sanitizers_experts_cpu.py builds and runs it):
 * argument errors of every entry point, sizes and addresses at their limits, and the choice of
 * kernel over drawn sizes. No call here reaches a launch: each fails a host-side check, has nothing to
 * do, or finds no device; as a second guard the program runs only where no GPU is
 * visible (exit 77 otherwise). Prints "host sanitize check ok" and exits 0 when every check holds. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gba_experts.h"

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

/* One call of each product with one size replaced. which: 0 T, 1 E, 2 N, 3 K. */
static int call(int op, int which, int64_t v, int act, int dtype, int flags, void *out, void *ws, size_t nb) {
    int64_t d[4] = {64, 4, 64, 64};
    if (which >= 0) d[which] = v;
    switch (op) {
    case GBX_FORWARD:
        return grouped_gemm_bias_act(at(1), at(2), at(3), at(4), out, at(6), d[0], d[1], d[2], d[3], act, dtype, flags, ws, nb);
    case GBX_ACT_GRAD:
        return grouped_gemm_act_grad(at(1), at(2), at(3), at(4), out, d[0], d[1], d[2], d[3], act, dtype, flags, ws, nb);
    case GBX_WGRAD:
        return grouped_gemm_wgrad(at(1), at(2), at(3), out, at(5), d[0], d[1], d[2], d[3], dtype, flags, ws, nb);
    case GBX_MX4:
        return grouped_gemm_bias_act_mx4(at(1), at(2), at(3), at(4), at(5), at(6), out, d[0], d[1], d[2], d[3], act, dtype, ws, nb);
    default:
        return gemm_bias_act_mx4(at(1), at(2), at(4), at(5), at(6), out, d[0], d[2], d[3], act, dtype, ws, nb);
    }
}

static void argument_errors(void) {
    const int ops[] = {GBX_FORWARD, GBX_ACT_GRAD, GBX_WGRAD, GBX_MX4, 5};
    for (int i = 0; i < 5; ++i) {
        const int op = ops[i];
        CHECK(call(op, -1, 0, 3, 0, 0, at(9), NULL, 0) == GBA_ERR_DEVICE);
        CHECK(call(op, -1, 0, 3, 7, 0, at(9), NULL, 0) == GBA_ERR_DTYPE);
        if (op != GBX_WGRAD) CHECK(call(op, -1, 0, -3, 0, 0, at(9), NULL, 0) == GBA_ERR_ACT);
        if (op < GBX_MX4) CHECK(call(op, -1, 0, 3, 0, 1 << 30, at(9), NULL, 0) == GBA_ERR_SHAPE);
        CHECK(call(op, -1, 0, 3, 0, 0, NULL, NULL, 0) == GBA_ERR_NULL);
        CHECK(call(op, -1, 0, 3, 0, 0, (char *)at(9) + 2, NULL, 0) == GBA_ERR_ALIGN);
        CHECK(call(op, -1, 0, 3, 0, 0, at(1), NULL, 0) == GBA_ERR_ALIAS);
        CHECK(call(op, -1, 0, 3, 0, 0, at(9), at(1), SIZE_MAX) == GBA_ERR_ALIAS);
        CHECK(call(op, -1, 0, 3, 0, 0, at(9), (void *)16, SIZE_MAX) == GBA_ERR_ALIAS);
        CHECK(call(op, -1, 0, 3, 0, 0, (void *)(UINTPTR_MAX - 15), NULL, 0) == GBA_ERR_DEVICE);
        for (int w = 0; w < 4; ++w)
            for (unsigned k = 0; k < sizeof kBad / sizeof *kBad; ++k)
                if (!(op == 5 && w == 1)) CHECK(call(op, w, kBad[k], 3, 0, 0, at(9), NULL, 0) == GBA_ERR_SHAPE);
        CHECK(call(op, 0, 0, 3, 0, 0, at(9), NULL, 0) == (op == GBX_WGRAD ? GBA_ERR_DEVICE : GBA_OK));   /* zeros to write */
        CHECK(call(op, 2, 0, 3, 0, 0, at(9), NULL, 0) == (op == GBX_ACT_GRAD ? GBA_ERR_DEVICE : GBA_OK));
        /* the largest sizes of each kind, whose products come near 2^62 bytes */
        CHECK(call(op, 0, (int64_t)1 << 29, 3, 0, 0, at(1), NULL, 0) == GBA_ERR_ALIAS);
        CHECK(call(op, 2, (int64_t)1 << 21, 3, 0, 0, at(1), NULL, 0) == GBA_ERR_ALIAS);
        CHECK(call(op, 3, (int64_t)1 << 21, 3, 0, 0, at(1), NULL, 0) == GBA_ERR_ALIAS);
    }
    CHECK(grouped_gemm_wgrad(at(1), at(2), at(3), at(4), at(5), 64, 4, 64, 64, 0, GBX_ACCUMULATE, NULL, 0) == GBA_ERR_DTYPE);
    for (int inverse = 0; inverse < 2; ++inverse) {
#define QUANT(X, C, S, M, K, D) (inverse ? mx4_dequantize(C, S, X, M, K, D) : mx4_quantize(X, C, S, M, K, D))
        CHECK(QUANT(at(1), at(2), at(3), 4, 64, 0) == GBA_ERR_DEVICE);
        CHECK(QUANT(at(1), at(2), at(3), 4, 64, -1) == GBA_ERR_DTYPE);
        CHECK(QUANT(at(1), at(2), at(3), 4, 48, 0) == GBA_ERR_ALIGN);
        CHECK(QUANT(NULL, at(2), at(3), 4, 64, 0) == GBA_ERR_NULL);
        CHECK(QUANT(at(1), at(1), at(3), 4, 64, 0) == GBA_ERR_ALIAS);
        CHECK(QUANT(at(1), at(2), at(3), INT32_MAX, 1 << 10, 0) == GBA_ERR_DEVICE);
        for (unsigned k = 0; k < sizeof kBad / sizeof *kBad; ++k) {
            CHECK(QUANT(at(1), at(2), at(3), kBad[k], 64, 0) == GBA_ERR_SHAPE);
            CHECK(QUANT(at(1), at(2), at(3), 4, kBad[k], 0) == GBA_ERR_SHAPE);
        }
    }
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
    gbx_plan p;
    for (int i = 0; i < 200000; ++i) {
        const int op = (int)(rnd() % 5);
        const int64_t T = spread(29), E = spread(12), N = (spread(18) + 7) / 8 * 8, K = spread(16) * 32;
        memset(&p, 0xff, sizeof p);
        const int s = gbx_get_plan(op, T, E, N, K, (size_t)spread(62), (int)spread(12), &p);
        CHECK(s == GBA_OK || (s == GBA_ERR_SHAPE && (op == GBX_ACT_GRAD ? N : K) > ((int64_t)1 << 21)));
        if (s == GBA_OK)
            CHECK(p.tile_m >= 16 && p.tile_m <= 256 && p.tile_n >= 64 && p.tile_n <= 256 && p.splits >= 1 && p.splits <= 16);
    }
    CHECK(gbx_get_plan(0, 1, 1, 8, 8, SIZE_MAX, INT32_MAX, &p) == GBA_OK);
    CHECK(gbx_get_plan(0, 1, 1, 8, 8, 0, 1, NULL) == GBA_ERR_NULL);
    for (int op = -1; op < 6; ++op)
        for (unsigned k = 0; k < sizeof kBad / sizeof *kBad; ++k) CHECK(gbx_get_plan(op, 1, 1, 8, kBad[k], 0, 256, &p) == GBA_ERR_SHAPE);
}

int main(void) {
    int ndev = 0;
    if (hipGetDeviceCount(&ndev) == 0 && ndev > 0) {
        printf("a GPU is visible: this check runs only without one\n");
        return 77;
    }
    CHECK(strlen(gbx_version()) > 0 && gbx_set_stream(NULL) == GBA_OK);
    argument_errors();
    plans();
    if (g_fail) {
        fprintf(stderr, "host sanitize check: FAILED\n");
        return 1;
    }
    printf("host sanitize check ok\n");
    return 0;
}
