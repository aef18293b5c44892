// Runs the kernels' search for experts and row tiles (gx_groups.hpp) on the CPU, by a wave of 64
// coroutines in lock step, for offsets of every kind: every tile that it names has to lie in its
// expert's rows, and those in the arrays, whatever the offsets hold. Built with the signed
// overflow check by tests/test_experts_groups_cpu.py. Prints "groups check ok" at the end.
#include <limits.h>
#include <stdio.h>
#include <stdlib.h>
#include <ucontext.h>

#include <algorithm>
#include <random>
#include <vector>

// ---- a wave: each lane operation is an exchange of one value a lane ----
namespace wave {
constexpr int kLanes = 64;
ucontext_t main_ctx, ctx[kLanes];
std::vector<char> stacks(kLanes << 16);
long long slot[kLanes], snap[kLanes];
int what[kLanes], cur, done;
void (*body)(int lane);

void entry() {
    body(cur);
    ++done;
    what[cur] = 0;
    swapcontext(&ctx[cur], &main_ctx);
}
// All lanes arrive with the same operation; then each sees what the others brought.
void exchange(int op, long long v) {
    slot[cur] = v;
    what[cur] = op;
    swapcontext(&ctx[cur], &main_ctx);
}
void run(void (*f)(int)) {
    body = f;
    done = 0;
    for (int l = 0; l < kLanes; ++l) {
        getcontext(&ctx[l]);
        ctx[l].uc_stack.ss_sp = &stacks[(size_t)l << 16];
        ctx[l].uc_stack.ss_size = 1 << 16;
        ctx[l].uc_link = &main_ctx;
        makecontext(&ctx[l], entry, 0);
    }
    while (done < kLanes) {
        for (cur = 0; cur < kLanes; ++cur) swapcontext(&main_ctx, &ctx[cur]);
        for (int l = 1; l < kLanes; ++l)
            if (what[l] != what[0]) {
                fprintf(stderr, "lanes part ways\n");
                exit(1);
            }
        std::copy(slot, slot + kLanes, snap);
    }
}
}  // namespace wave

template <class T>
T __shfl_up(T v, int d) {
    const int l = wave::cur;
    wave::exchange(1, v);
    return l >= d ? (T)wave::snap[l - d] : v;
}
template <class T>
T __shfl_xor(T v, int d) {
    const int l = wave::cur;
    wave::exchange(2, v);
    return (T)wave::snap[l ^ d];
}
unsigned long long __ballot(bool p) {
    wave::exchange(3, p);
    unsigned long long m = 0;
    for (int l = 0; l < wave::kLanes; ++l) m |= (unsigned long long)(wave::snap[l] != 0) << l;
    return m;
}
int lane_read(int v, int l) {
    if (l < 0 || l >= wave::kLanes) {
        fprintf(stderr, "reads lane %d\n", l);
        exit(1);
    }
    wave::exchange(4 + l, v);   // the same lane for all of them
    return (int)wave::snap[l];
}
#define __builtin_amdgcn_readlane lane_read
#define __builtin_amdgcn_readfirstlane(v) lane_read(v, 0)
int __ffsll(unsigned long long m) { return m ? __builtin_ctzll(m) + 1 : 0; }
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
namespace gba {
constexpr int ceil_div(int x, int b) { return (int)(((long long)x + b - 1) / b); }
}  // namespace gba

#include "gx_groups.hpp"

// ---- the check ----
using namespace gbx;

static Group g;
static int bm, wanted, totals[64];
static Found found[64];
static bool few_way;

// What a workgroup does (gx_ring.hpp; the persistent kernel with few_row_tile).
static void search(int lane) {
    if (g.E <= 64 && few_way) {
        int start = 0, rows = 0;
        if (lane < g.E) expert_rows(g, lane, start, rows);
        const int upto = wave_scan(gba::ceil_div(rows, bm), lane);
        totals[lane] = min(__builtin_amdgcn_readlane(upto, 63), g.row_bound);
        if (wanted >= 0 && wanted < totals[lane]) found[lane] = few_row_tile(upto, start, rows, wanted);
    } else if (g.E <= 64) {
        found[lane] = locate_few(g, bm, lane, [&](int total) {
            totals[lane] = total;
            return wanted < total ? wanted : -1;
        });
    } else {
        totals[lane] = total_row_tiles(g, bm, lane);
        if (wanted >= 0 && wanted < totals[lane]) found[lane] = find_row_tile(g, bm, wanted, lane);
    }
}

static long long tiles_checked;

#define CHECK(cond)                                                                                          \
    do {                                                                                                     \
        if (!(cond)) {                                                                                       \
            fprintf(stderr, "%s: %s, T %d, E %d, tile rows %d, tile %d\n", name, #cond, g.T, g.E, bm, wanted); \
            exit(1);                                                                                         \
        }                                                                                                    \
    } while (0)

static int clamped(int v) { return v < 0 ? 0 : v > g.T ? g.T : v; }

static void check(const char *name, const std::vector<int> &offsets, int T, int tile_rows, std::mt19937 &rng) {
    bm = tile_rows;
    g = Group();
    g.T = T;
    g.E = (int)offsets.size() - 1;
    g.offsets = offsets.data();
    g.row_bound = (int)row_tile_bound(T, g.E, bm);
    // The tiles before each expert, in 64 bits.
    std::vector<long long> before(1, 0);
    bool sorted = true;
    for (int e = 0; e < g.E; ++e) {
        const long long n = std::max((long long)clamped(offsets[e + 1]) - clamped(offsets[e]), 0LL);
        sorted &= clamped(offsets[e + 1]) >= clamped(offsets[e]);
        before.push_back(before.back() + (n + bm - 1) / bm);
    }
    const long long all = before.back(), total = std::min(all, (long long)g.row_bound);
    wanted = -1;
    CHECK(!sorted || all <= g.row_bound);   // the grid holds every tile of offsets in order
    const int ways = g.E <= 64 ? 2 : 1;
    for (int way = 0; way < ways; ++way) {
        few_way = way == 1;
        // First, last and past it, the ends of some experts, and some in between.
        std::vector<long long> some = {-1, 0, 1, total - 2, total - 1, total, total + 1};
        for (int k = 0; k < (g.E > 200 ? 2 : g.E > 64 ? 4 : 8); ++k) {
            some.push_back(before[rng() % (g.E + 1)]);
            some.push_back(before[rng() % (g.E + 1)] - 1);
            if (total > 0) some.push_back((long long)(rng() % total));
        }
        for (long long t : some) {
            if (t < -1 || t > INT_MAX) continue;
            wanted = (int)t;
            for (Found &f : found) f = Found{-7, -7, -7, -7, -7, -7};
            wave::run(search);
            for (int l = 0; l < 64; ++l) {
                CHECK(totals[l] == total);
                if (t < 0 || t >= total) continue;
                const Found &f = found[l];
                CHECK(f.e >= 0 && f.e < g.E);
                CHECK(f.start == clamped(offsets[f.e]) && f.start >= 0);
                CHECK(f.rows == clamped(offsets[f.e + 1]) - f.start && f.rows > 0 && f.start + f.rows <= T);
                CHECK(f.before == before[f.e] && f.tiles == (f.rows + bm - 1) / bm);
                CHECK(t >= f.before && t < (long long)f.before + f.tiles);
                CHECK((t - f.before) * bm < f.rows);   // the tile's first row is one of the expert's
            }
            tiles_checked += t >= 0 && t < total;
        }
    }
}

int main() {
    std::mt19937 rng(7);
    for (int T : {1, 40, 1000, 1 << 29})
        for (int E : {1, 2, 63, 64, 65, 200, 4096})
            for (int rows : {16, 256}) {
                const int n = E + 1;
                std::vector<int> o(n);
                auto fill = [&](auto &&f) {
                    for (int i = 0; i < n; ++i) o[i] = f(i);
                };
                auto any = [&] { return (int)rng(); };
                auto inside = [&] { return (int)(rng() % ((unsigned)T + 1)); };
                fill([&](int) { return inside(); });
                std::sort(o.begin(), o.end());
                check("in order", o, T, rows, rng);
                std::reverse(o.begin(), o.end());
                check("in reverse order", o, T, rows, rng);
                fill([&](int) { return inside(); });
                check("in no order", o, T, rows, rng);
                fill([&](int i) { return i % 2 ? T : 0; });
                check("nothing and everything in turn", o, T, rows, rng);
                fill([&](int i) { return i % 2 ? INT_MAX : INT_MIN; });
                check("the type's ends in turn", o, T, rows, rng);
                fill([&](int) { return any(); });
                check("anything", o, T, rows, rng);
                std::sort(o.begin(), o.end());
                check("anything in order", o, T, rows, rng);
                fill([&](int) { return INT_MAX; });
                check("all past the end", o, T, rows, rng);
                fill([&](int) { return INT_MIN; });
                check("all before the start", o, T, rows, rng);
                fill([&](int i) { return i == 0 ? INT_MIN : INT_MAX; });
                check("one expert with everything", o, T, rows, rng);
                fill([&](int i) { return i == n - 1 ? T : 0; });
                check("the last with everything", o, T, rows, rng);
                if (T < 1000 && E <= 65) {   // groups of one and two rows
                    fill([&](int i) { return i == 0 ? 0 : o[i - 1] + (int)(rng() % 3); });
                    check("short", o, T, rows, rng);
                }
            }
    // No offsets: one expert with all rows.
    g = Group();
    g.T = 77;
    g.E = 1;
    int start = -1, count = -1;
    expert_rows(g, 0, start, count);
    if (start != 0 || count != 77) return 1;
    printf("groups check ok, %lld tiles\n", tiles_checked);
    return 0;
}
