// The groups of a grouped product, and the search for the expert and row tile of a work
// unit. Offsets come from device memory and may hold anything: the clamps and the bound on the
// tiles here are what keeps every tile inside its expert's rows. Nothing but the lane
// operations of a wave is used, so that a host program can run this code with a wave of its own
// (ceil_div of gba_kernels.hpp, min and max are the includer's).
#pragma once

#include <stdint.h>

namespace gbx {

using namespace gba;

// A grouped product. Rows mode: the rows of expert e of A [T][K] times B_e, giving rows of
// C [T][N]. Weight gradients: At_e^T.B_e over the rows of expert e, with At [T][M]
// and B [T][N], giving C [E][M][N]. K counts 16-bit words.
struct Group {
    const uint16_t *A, *B;
    const uint32_t *sa, *sb;     // MX4 scale planes of A and B, one dword a row; F8: fp32, planes of A, blocks
                                 // of B [E][N / 128][K / 128] (rounded up)
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

// First row and row count of an expert from its two offsets, clamped to [0, T]: whatever they
// hold, start + rows <= T.
__device__ __forceinline__ void rows_between(int lo, int hi, int T, int &start, int &rows) {
    start = clamp_row(lo, T);
    rows = max(clamp_row(hi, T) - start, 0);
}

// Those of expert e.
__device__ __forceinline__ void expert_rows(const Group &g, int e, int &start, int &rows) {
    if (!g.offsets) {
        start = 0;
        rows = g.T;
        return;
    }
    rows_between(g.offsets[e], g.offsets[e + 1], g.T, start, rows);
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

// The same from one register a lane (up to 64 experts, lane l's: the row tiles of experts 0 .. l, the
// first row and the rows of expert l), for a tile that is there.
__device__ __forceinline__ Found few_row_tile(int upto, int start, int rows, int t) {
    const unsigned long long past = __ballot(upto > t);
    Found f;
    f.e = __builtin_amdgcn_readfirstlane(__ffsll(past) - 1);
    f.before = f.e > 0 ? __builtin_amdgcn_readlane(upto, f.e - 1) : 0;
    f.tiles = __builtin_amdgcn_readlane(upto, f.e) - f.before;
    f.start = __builtin_amdgcn_readlane(start, f.e);
    f.rows = __builtin_amdgcn_readlane(rows, f.e);
    f.total = 0;
    return f;
}

}  // namespace gbx
