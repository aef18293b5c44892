// Tile kernel of the grouped products: one BM x BN tile of one expert's output
// per workgroup, K walked in 64-word slices (128 bytes a row) through a ring of
// LDS stages that direct-to-LDS loads fill STAGES - 1 slices ahead.
//
// A workgroup finds its expert itself: the row tiles of all experts are counted
// from the offsets in device memory (a wave scan, redone by every wave), so the
// host needs no copy of them. The grid is the most tiles T rows can make; the
// workgroups past the last tile end at once.
//
// Operand layouts: K-contiguous rows (A; B with TB) and rows along K (B [K][N]
// without TB; At [T][M] with TA), in LDS as in gemm_v3.hpp, chunks XOR-swizzled so that
// the fragment reads have no bank conflicts. Edges cost no branches: rows past
// the expert's end, columns past N and words past K read as zeros (buffer range
// checks and out-of-range offsets).
//
// What bounds it: with few rows an expert, HBM (each weight is read once: 16 rows on
// 12 of 32 experts of 2816 x 2048 bf16 take 23 us, 6.0 TB/s; 5 x 14336 x 4096 in 4
// bits 8.5 us, 3.7 TB/s, 16 slices being mostly latency); with tens of rows, loads and
// matrix instructions about equally (999 rows on 15 experts, 1408 x 2048 fp16: 19 to 23 us by
// their shares, 250 to 300 TFLOP/s). 128 x 128 is the largest tile of which two workgroups share a CU; larger
// products are the persistent kernel's.
#pragma once

#include "gx_common.hpp"

namespace gbx {

// buffer_load_lds16 (gba_dma.hpp), non-temporal.
__device__ __forceinline__ void buffer_load_lds16_nt(__amdgpu_buffer_rsrc_t rsrc, uint32_t voffset, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, 0 offen nt lds"
        :
        : "v"(voffset), "s"(rsrc), "s"(lds_base)
        : "memory", "m0");
}

template <int BM, int BN, int WM, int WN, int STAGES, int OP, int ODT, int EPI, bool TB, bool TA>
__global__ void __launch_bounds__(256, 2)   // two workgroups a CU at least
grouped_ring_kernel(Group g) {
    constexpr int NT = 256, BK = 64;
    constexpr bool MX = OP == OP_MX4, F8 = OP == OP_F8;
    constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    constexpr int CHT = BM / 8, CHB = BN / 8;   // chunks per k row of At's and B's tiles
    constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    // MX4: a slice's scales, 2 planes of one dword a row for A, then for B. F8: A's plane.
    constexpr int S_BYTES = MX ? 8 * (BM + BN) : F8 ? 4 * BM : 0;
    constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES;
    // Loads of a slice per thread. A tile of fewer than 256 chunks is loaded
    // by every group of waves that it fills, the same bytes to the same place.
    constexpr int A_LD = BM * 8 >= NT ? BM * 8 / NT : 1, B_LD = BN * 8 / NT;
    constexpr int AW = BM * 8 >= NT ? 4 : BM * 8 / 64;   // waves that a load of A fills
    constexpr int LD = A_LD + B_LD + (MX || F8 ? 1 : 0);
    static_assert(WM * WN == 4 && WTM % 16 == 0 && WTN % 16 == 0, "four waves of whole MFMA blocks");
    static_assert(BN * 8 % NT == 0 && (BM * 8 % NT == 0 || NT % (BM * 8) == 0), "loads split evenly");
    static_assert(!TA || (CHT >= 8 && !TB && !MX), "At: 64 rows or more");
    static_assert(TB || CHB >= 8, "B swizzle needs 8 chunks per row");
    static_assert(!MX || (TB && BM <= 256 && BN <= 256), "4-bit operands are K-contiguous");
    static_assert(!F8 || (TB && !TA && BM >= 16 && BM <= 1024 && 128 % BN == 0), "8-bit operands: K-contiguous, one block of B's columns");
    static_assert(STAGES * STAGE <= 160 * 1024 && (STAGES - 1) * LD < 64, "ring");

    __shared__ __attribute__((aligned(1024))) char smem[STAGES * STAGE];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wid / WN, wn = wid % WN;

    // ---- the work unit: expert, tile, K range ----
    const int tiles_n = ceil_div(g.N, BN);
    int e, start, rows, m0, n0, split = 0;
    {
        const long long b = (long long)blockIdx.y * gridDim.x + blockIdx.x;
        // This workgroup's tile among `tiles` (split-major units, one contiguous range an XCD), or -1.
        auto my_tile = [&](long long tiles) __attribute__((always_inline)) {
            const long long units = tiles * g.splits;
            if (b >= units) return -1;
            const int u = xcd_remap((int)b, (int)units);
            split = u / (int)tiles;
            return u - split * (int)tiles;
        };
        int tm, tn;
        if constexpr (TA) {
            const int tiles_m = ceil_div(g.M, BM);
            const int u = my_tile((long long)g.E * tiles_m * tiles_n);
            if (u < 0) return;
            e = u / (tiles_m * tiles_n);
            grouped_tile(u - e * tiles_m * tiles_n, tiles_m, tiles_n, 4, tm, tn);
            expert_rows_uniform(g, e, start, rows);
        } else {
            int u = -1;
            Found f;
            if (g.E <= 64) {
                f = locate_few(g, BM, lane, [&](int total) __attribute__((always_inline)) {
                    u = my_tile((long long)total * tiles_n);
                    return u < 0 ? -1 : u / tiles_n;
                });
                if (u < 0) return;
            } else {
                u = my_tile((long long)total_row_tiles(g, BM, lane) * tiles_n);
                if (u < 0) return;
                f = find_row_tile(g, BM, u / tiles_n, lane);
            }
            e = f.e;
            start = f.start;
            rows = f.rows;
            grouped_tile(u - f.before * tiles_n, max(f.tiles, 1), tiles_n, 4, tm, tn);
        }
        m0 = tm * BM;
        n0 = tn * BN;
        // Offsets that decrease could name a tile past its expert's rows.
        if (!TA && (m0 < 0 || m0 >= rows || n0 < 0)) return;
    }
    const int K = TA ? rows : g.K;          // depth of the sum
    const int M = TA ? g.M : rows;          // rows of the expert's output
    const int N = g.N;
    const int nk_all = ceil_div(K, BK);
    const int kt0 = (int)((long long)split * nk_all / g.splits);
    const int nk = (int)((long long)(split + 1) * nk_all / g.splits) - kt0;
    const int rows_a = min(M - m0, BM), rows_b = min(N - n0, BN);
    const uint16_t *const Ae = g.A + (TA ? (size_t)start * M : (size_t)start * K);
    const uint16_t *const Be = TA ? g.B + (size_t)start * N : g.B + (size_t)e * K * N;

    // ---- loads ----
    // Byte offsets from a slice's corner, which the descriptor carries. Load i of
    // a K-contiguous tile: row i*32 + tid/8, chunk (tid%8) ^ (row%8); of a tile
    // with rows along K: k row, chunk ^ bswz(k row), columns past the edge out of range.
    uint32_t off[A_LD + B_LD];
    const int ta = tid & (AW * 64 - 1);
    const int ca = (tid & 7) ^ ((tid >> 3) & 7);   // chunk of every K-contiguous load
#pragma unroll
    for (int i = 0; i < A_LD; ++i) {
        const int s = i * NT + ta;
        if constexpr (TA) {
            const int r = s / CHT, c = (s % CHT) ^ bswz<CHT>(r);
            off[i] = m0 + c * 8 < M ? (uint32_t)r * (uint32_t)M * 2u + (uint32_t)c * 16u : kOobOffset;
        } else {
            off[i] = (uint32_t)(s >> 3) * (uint32_t)K * 2u + (uint32_t)ca * 16u;
        }
    }
#pragma unroll
    for (int i = 0; i < B_LD; ++i) {
        const int s = i * NT + tid;
        if constexpr (TB) {
            off[A_LD + i] = (uint32_t)(s >> 3) * (uint32_t)K * 2u + (uint32_t)ca * 16u;
        } else {
            const int r = s / CHB, c = (s % CHB) ^ bswz<CHB>(r);
            off[A_LD + i] = n0 + c * 8 < N ? (uint32_t)r * (uint32_t)N * 2u + (uint32_t)c * 16u : kOobOffset;
        }
    }
    const uint32_t smem_lds = (uint32_t)(uintptr_t)(GBA_LDS void *)smem;
    const bool stream = (g.flags & GF_STREAM) != 0;
    auto load_b = [&](__amdgpu_buffer_rsrc_t rsrc, uint32_t voffset, uint32_t dst) __attribute__((always_inline)) {
        if (BM <= 64 && stream)
            buffer_load_lds16_nt(rsrc, voffset, dst);
        else
            buffer_load_lds16(rsrc, voffset, dst);
    };
    // The slice to load next: its corners and byte ranges, carried from slice to
    // slice. Up to the last slice they move by constants; the last one (K's end:
    // chunks past it out of range, fewer rows) and those past it (empty ranges: zeros land
    // and no memory is read, which keeps the wait counts uniform) are formed in
    // one rarely taken block. Forming every slice from scratch cost a wave that has its
    // SIMD to itself as long as the slice's matrix work.
    struct {
        const uint16_t *pa, *pb;
        uint32_t na, nb;
        const uint32_t *ps;   // MX4: this wave's scale plane: w % 2 of A's (w < 2) or B's. F8: A's
        uint32_t ns;
        int left;             // slices left to load
    } pos;
    const size_t plane_dwords = MX ? (wid < 2 ? (size_t)g.T : (size_t)g.E * N) : 0;
    auto at_end = [&](int kt) __attribute__((always_inline)) {
        const int k0 = (kt0 + kt) * BK;
        const uint32_t kin = pos.left > 0 ? (uint32_t)min(K - k0, BK) : 0u;
        if constexpr (TA) {
            pos.na = kin * (uint32_t)M * 2u;
        } else {
            if (pos.left <= 0) pos.na = 0;
#pragma unroll
            for (int i = 0; i < A_LD; ++i)
                if ((uint32_t)ca * 8u >= kin) off[i] = kOobOffset;
        }
        if constexpr (!TB) {
            pos.nb = kin * (uint32_t)N * 2u;
        } else {
            if (pos.left <= 0) pos.nb = 0;
#pragma unroll
            for (int i = 0; i < B_LD; ++i)
                if ((uint32_t)ca * 8u >= kin) off[A_LD + i] = kOobOffset;
        }
        // 32 words: 128 values a plane
        if (MX && (pos.left <= 0 || (2 * (kt0 + kt) + (wid & 1)) * 32 >= K)) pos.ns = 0;
        if (F8 && pos.left <= 0) pos.ns = 0;
    };
    {
        const int k0 = kt0 * BK;
        if constexpr (TA) {
            pos.pa = Ae + ((size_t)k0 * M + m0);
            pos.na = (uint32_t)BK * (uint32_t)M * 2u;
        } else {
            pos.pa = Ae + ((size_t)m0 * K + k0);
            pos.na = (uint32_t)rows_a * (uint32_t)K * 2u - (uint32_t)k0 * 2u;
        }
        if constexpr (TB) {
            pos.pb = Be + ((size_t)n0 * K + k0);
            pos.nb = (uint32_t)rows_b * (uint32_t)K * 2u - (uint32_t)k0 * 2u;
        } else {
            pos.pb = Be + ((size_t)k0 * N + n0);
            pos.nb = (uint32_t)BK * (uint32_t)N * 2u;
        }
        pos.left = nk;
        if constexpr (MX) {
            pos.ps = (wid < 2 ? g.sa + (size_t)start + m0 : g.sb + (size_t)e * N + n0) +
                     (size_t)(2 * kt0 + (wid & 1)) * plane_dwords;
            pos.ns = (uint32_t)(wid < 2 ? rows_a : rows_b) * 4u;
        }
        if constexpr (F8) {
            pos.ps = g.sa + (size_t)kt0 * g.T + start + m0;
            pos.ns = (uint32_t)rows_a * 4u;
        }
    }
    // Loads the next slice, which is slice kt of this unit, into stage S.
    auto load_slice = [&](int kt, auto stage_c) __attribute__((always_inline)) {
        constexpr int S = decltype(stage_c)::value;
        if (__builtin_expect(pos.left <= 1, 0)) at_end(kt);
        const uint32_t base = smem_lds + (uint32_t)(S * STAGE);
        const __amdgpu_buffer_rsrc_t ra = make_rsrc(pos.pa, pos.na), rb = make_rsrc(pos.pb, pos.nb);
        const uint32_t wave_a = base + (uint32_t)((wid & (AW - 1)) * 1024);
#pragma unroll
        for (int i = 0; i < A_LD; ++i) buffer_load_lds16(ra, off[i], wave_a + (uint32_t)(i * NT * 16));
#pragma unroll
        for (int i = 0; i < B_LD; ++i)
            load_b(rb, off[A_LD + i], base + (uint32_t)(A_BYTES + wid * 1024 + i * NT * 16));
        if constexpr (MX) {
            // Four rows' dwords a lane (range checks are per dword); the lanes past
            // the tile's rows are switched off.
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(pos.ps, pos.ns);
            const uint32_t dst = base + (uint32_t)(A_BYTES + B_BYTES) +
                                 (wid < 2 ? (uint32_t)((wid & 1) * BM * 4) : (uint32_t)(2 * BM * 4 + (wid & 1) * BN * 4));
            if (lane * 4 < (wid < 2 ? BM : BN)) buffer_load_lds16(rs, (uint32_t)lane * 16u, dst);
            pos.ps += 2 * plane_dwords;
        }
        if constexpr (F8) {
            // A quarter of the tile's rows a wave, one lane of it at least.
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(pos.ps, pos.ns);
            if (lane * 16 < BM) buffer_load_lds16(rs, (uint32_t)(wid * BM + lane * 16), base + (uint32_t)(A_BYTES + B_BYTES + wid * BM));
            pos.ps += g.T;
        }
        if constexpr (TA) {
            pos.pa += (size_t)BK * M;
        } else {
            pos.pa += BK;
            pos.na -= 2u * BK;
        }
        if constexpr (TB) {
            pos.pb += BK;
            pos.nb -= 2u * BK;
        } else {
            pos.pb += (size_t)BK * N;
        }
        --pos.left;
    };

    // ---- fragments ----
    const int tg = lane >> 4, tj = lane & 15;
    f32x4 acc[FN][FM];
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int b = 0; b < FM; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Frags {
        u32x4 a[FM], b[FN];
        uint32_t sa[FM], sb[FN];
    };
    // Rows along K are gathered by transposing reads of four k rows each.
    auto gather = [&](const char *tile, int kk, int x, int row_bytes, auto chunks_c) __attribute__((always_inline)) {
        constexpr int CHUNKS = decltype(chunks_c)::value;
        i16x4 h[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = kk * 32 + 8 * tg + 4 * i + (tj >> 2);
            h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (GBA_LDS i16x4 *)(tile + k * row_bytes + (((x >> 3) ^ bswz<CHUNKS>(k)) * 16) + (x & 4) * 2));
        }
        return __builtin_bit_cast(u32x4, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto read_frags = [&](const char *base, int kk, Frags &f) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < FM; ++b) {
            if constexpr (TA) {
                f.a[b] = gather(base, kk, wm * WTM + b * 16 + 4 * (tj & 3), BM * 2, std::integral_constant<int, CHT>{});
            } else {
                const int r = wm * WTM + b * 16 + tj;
                f.a[b] = *reinterpret_cast<const u32x4 *>(base + r * 128 + (((4 * kk + tg) ^ (r & 7)) * 16));
            }
            if constexpr (MX)
                f.sa[b] = *reinterpret_cast<const uint32_t *>(base + A_BYTES + B_BYTES + kk * BM * 4 +
                                                              (wm * WTM + b * 16 + tj) * 4) >> (8 * tg);
        }
#pragma unroll
        for (int a = 0; a < FN; ++a) {
            if constexpr (TB) {
                const int r = wn * WTN + a * 16 + tj;
                f.b[a] = *reinterpret_cast<const u32x4 *>(base + A_BYTES + r * 128 + (((4 * kk + tg) ^ (r & 7)) * 16));
            } else {
                f.b[a] = gather(base + A_BYTES, kk, wn * WTN + a * 16 + 4 * (tj & 3), BN * 2,
                                std::integral_constant<int, CHB>{});
            }
            if constexpr (MX)
                f.sb[a] = *reinterpret_cast<const uint32_t *>(base + A_BYTES + B_BYTES + 2 * BM * 4 + kk * BN * 4 +
                                                              (wn * WTN + a * 16 + tj) * 4) >> (8 * tg);
        }
    };
    auto multiply = [&](const Frags &f) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < FN; ++a)
#pragma unroll
            for (int b = 0; b < FM; ++b) {
                if constexpr (MX)
                    acc[a][b] = mfma_mx4(f.b[a], f.a[b], acc[a][b], f.sb[a], f.sa[b]);
                else if constexpr (!F8)
                    acc[a][b] = mfma16x16x32<OP>(f.b[a], f.a[b], acc[a][b]);
            }
    };

    // F8: one matrix instruction is one block of K. Its sums are scaled as they are added: by A's scale of the row
    // (a lane's four sums share a row) times B's of the tile's columns, which comes by a scalar load a slice
    // ahead. The 128 values lie across the lanes as chunks tg and 4 + tg, in both operands alike.
    typedef const float __attribute__((address_space(4))) *ScalePtr;
    ScalePtr wscales = nullptr;
    float wscale = 0.f, wscale_next = 0.f;
    if constexpr (F8) {
        const int blocks = ceil_div(K, BK);
        wscales = (ScalePtr)(uintptr_t)((const float *)g.sb + ((size_t)e * ceil_div(N, 128) + n0 / 128) * blocks + kt0);
        if (nk > 0) wscale_next = wscales[0];
    }
    auto multiply_f8 = [&](const char *base, const Frags &f0, const Frags &f1) __attribute__((always_inline)) {
        const auto both = [](const u32x4 &x, const u32x4 &y) __attribute__((always_inline)) {
            return i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
        };
        float s[FM];
#pragma unroll
        for (int b = 0; b < FM; ++b)
            s[b] = *reinterpret_cast<const float *>(base + A_BYTES + B_BYTES + (wm * WTM + b * 16 + tj) * 4) * wscale;
#pragma unroll
        for (int a = 0; a < FN; ++a)
#pragma unroll
            for (int b = 0; b < FM; ++b) {
                const f32x4 p = mfma_f8(both(f0.b[a], f1.b[a]), both(f0.a[b], f1.a[b]));
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[a][b][i] = fmaf(p[i], s[b], acc[a][b][i]);
            }
    };

    // ---- the slices ----
    static_for<STAGES - 1>([&](auto s_c) __attribute__((always_inline)) { load_slice(decltype(s_c)::value, s_c); });
    // Slice kt lies in stage kt % STAGES, a constant in each copy of the loop's body.
    for (int kb = 0; kb < nk; kb += STAGES) {
        static_for<STAGES>([&](auto s_c) __attribute__((always_inline)) {
            constexpr int S = decltype(s_c)::value;
            if (S == 0 || kb + S < nk) {
                // Slice kt has landed and this wave's reads of slice kt - 1 are done; then the
                // same holds for all waves, and slice kt - 1's stage is free.
                wait_vmcnt_lgkm0<(STAGES - 2) * LD>();
                block_barrier();
                const char *const base = smem + S * STAGE;
                if constexpr (F8) {
                    wscale = wscale_next;
                    wscale_next = wscales[min(kb + S + 1, nk - 1)];
                }
                constexpr std::integral_constant<int, (S + STAGES - 1) % STAGES> freed{};
                // A ring of two stages has its next slice only now to ask for: first of
                // all. Longer ones ask while their first fragments are on the way (small tiles
                // 5 to 20 % faster so, 128 x 128 15 % slower).
                if constexpr (F8) {
                    Frags f0, f1;
                    if constexpr (STAGES == 2) load_slice(kb + S + 1, freed);
                    read_frags(base, 0, f0);
                    read_frags(base, 1, f1);
                    if constexpr (STAGES > 2) load_slice(kb + S + STAGES - 1, freed);
                    multiply_f8(base, f0, f1);
                } else if constexpr (STAGES == 2) {
                    load_slice(kb + S + 1, freed);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        Frags f;
                        read_frags(base, kk, f);
                        multiply(f);
                    }
                } else {
                    Frags f0, f1;
                    read_frags(base, 0, f0);
                    load_slice(kb + S + STAGES - 1, freed);
                    read_frags(base, 1, f1);
                    multiply(f0);
                    multiply(f1);
                }
            }
        });
    }

    // ---- epilogue ----
    // The tile's fp32 sums go through the ring's LDS (a lane: one row, four adjacent
    // columns) to threads of eight adjacent columns, so that every global access of the
    // epilogue is 16 bytes a lane and whole 128-byte lines: writing a weight
    // gradient's tile from the matrix layout (32 bytes a row) took 1.6 times as long.
    // Chunk q (16 bytes) of row r lies at q ^ (r % 8).
    wait_vmcnt_lgkm0<0>();
    block_barrier();   // every wave's loads have landed and its reads are done
    constexpr int QN = BN / 4, TC = BN / 8, UNITS = BM * TC / NT > 0 ? BM * TC / NT : 1;
    static_assert(BM * BN * 4 <= STAGES * STAGE, "the sums fit the ring");
    static_assert(NT % TC == 0, "a thread keeps its columns");
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int b = 0; b < FM; ++b) {
            const int r = wm * WTM + b * 16 + tj, q = (wn * WTN + a * 16) / 4 + tg;
            *reinterpret_cast<f32x4 *>(smem + (r * QN + (q ^ (r & 7))) * 16) = acc[a][b];
        }
    wait_vmcnt_lgkm0<0>();
    block_barrier();
    const int col = tid % TC, n = n0 + col * 8;
    const size_t crow = TA ? (size_t)e * M : (size_t)start;
    // f(the eight sums of row m0 + r from column n on, their place in the output)
    auto each = [&](auto &&f) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int r = u * (NT / TC) + tid / TC;
            if (r >= rows_a || n >= N) continue;   // N is a multiple of 8
            const int q = 2 * col;
            f32x4 v[2] = {*reinterpret_cast<const f32x4 *>(smem + (r * QN + (q ^ (r & 7))) * 16),
                          *reinterpret_cast<const f32x4 *>(smem + (r * QN + ((q + 1) ^ (r & 7))) * 16)};
            f(v, (crow + m0 + r) * (size_t)N + n);
        }
    };
    if constexpr (EPI == EPI_PART) {
        float *const P = g.part + (size_t)split * (TA ? (size_t)g.E * M : (size_t)g.T) * N;
        each([&](f32x4 (&v)[2], size_t at) {
            *reinterpret_cast<f32x4 *>(P + at) = v[0];
            *reinterpret_cast<f32x4 *>(P + at + 4) = v[1];
        });
    } else {
        each([&](f32x4 (&v)[2], size_t at) { finish<EPI, ODT>(g, v, e, n, at); });
    }
}

template <int BM, int BN, int WM, int WN, int STAGES, int OP, int ODT, int EPI, bool TB, bool TA>
hipError_t launch_ring(Group g, hipStream_t stream) {
    const long long tiles_n = ceil_div(g.N, BN);
    const long long row_tiles = TA ? (long long)g.E * ceil_div(g.M, BM) : row_tile_bound(g.T, g.E, BM);
    const long long units = row_tiles * tiles_n * g.splits;
    if (units <= 0) return hipSuccess;
    if (units > 0x7fffffffLL - kGridX) return hipErrorInvalidValue;
    g.row_bound = (int)row_tiles;
    return launch(grouped_ring_kernel<BM, BN, WM, WN, STAGES, OP, ODT, EPI, TB, TA>, tile_grid(units), dim3(256), stream, g);
}

}  // namespace gbx
