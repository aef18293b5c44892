// Persistent kernel of the large 8-bit products: one workgroup per CU walks its 256 x 256
// tiles, over all experts, as one stream of K slices of 128 (one block) through a two-stage LDS
// ring.
//
// A slice's sums come out of the matrix cores alone (accumulator input 0) and are scaled as they are added:
// acc += sa[row] sw t, one vector instruction a value. Vector instructions reach 256 registers, so that a wave's
// accumulators are at most half of them: eight waves of 64 x 128 (two a SIMD), where the kernels without scales have
// four of 128 x 128 in accumulation registers. 32 matrix instructions a slice and wave (32 cycles each) then
// stand beside 128 multiply-adds (4 cycles), and the other wave of the SIMD fills what one leaves.
//
// A slice runs in four groups of two column blocks x four row blocks. While one group multiplies, the next one's
// column fragments are read. Before the last group everything of the slice is in registers: the waves meet
// (the next slice has landed, this one's stage is free), the loads of the slice after the next go out, and the
// next slice's first fragments are read as this one's row fragments are used up. A matrix instruction's sums are
// taken up LAG instructions later, the last ones in the next slice.
//
// Operands, swizzle and tiles as grouped_ring_kernel's; a lane's 32 values of a row are chunks tg and tg + 4.
#pragma once

#include "gm_common.hpp"
#include "../experts/gx_groups.hpp"
#include "gemm_v5.hpp"   // lane_now

namespace gbm {

using gbx::Group;
using gbx::Found;

// acc += t s (FIRST: acc = t s) on four values, kept where it stands (left to itself the compiler gathers a slice's
// multiply-adds at its end, with all its sums held). It places no waits between a matrix instruction and these
// reads of its sums: LAG matrix instructions, which cannot issue before the pipe takes them, 32 cycles each, lie between.
template <bool FIRST>
__device__ __forceinline__ void scaled_add(float (&acc)[4], const f32x4 &t, float s) {
    if constexpr (FIRST)
        asm volatile("v_mul_f32 %0, %4, %8\n\tv_mul_f32 %1, %5, %8\n\tv_mul_f32 %2, %6, %8\n\tv_mul_f32 %3, %7, %8"
                     : "=&v"(acc[0]), "=&v"(acc[1]), "=&v"(acc[2]), "=&v"(acc[3])
                     : "v"(t[0]), "v"(t[1]), "v"(t[2]), "v"(t[3]), "v"(s));
    else
        asm volatile("v_fmac_f32 %0, %4, %8\n\tv_fmac_f32 %1, %5, %8\n\tv_fmac_f32 %2, %6, %8\n\tv_fmac_f32 %3, %7, %8"
                     : "+&v"(acc[0]), "+&v"(acc[1]), "+&v"(acc[2]), "+&v"(acc[3])
                     : "v"(t[0]), "v"(t[1]), "v"(t[2]), "v"(t[3]), "v"(s));
}

// Loads one dword a lane: lane l's lands at LDS byte address lds_base + 4 l.
__device__ __forceinline__ void buffer_load_lds4(__amdgpu_buffer_rsrc_t rsrc, uint32_t voffset, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %0, %1, 0 offen lds"
        :
        : "v"(voffset), "s"(rsrc), "s"(lds_base)
        : "memory", "m0");
}

template <int ODT, int EPI, int ACT>
__global__ void __launch_bounds__(512, 2)
f8_persist_kernel(Group g) {
    constexpr int BM = 256, BN = 256, NW = 8, WTM = 64, WTN = 128, FM = 4, FN = 8, LAG = 3, NMF = FM * FN;
    constexpr int TILE = 32768, SCALES = 2 * TILE, STAGE = SCALES + 1024 + NW * 256;   // A, W, A's scales, a W scale a lane
    constexpr int STG = 16 * 64 * 2;   // epilogue: 16 rows x 64 columns a wave
    constexpr bool BIASED = EPI == gbx::EPI_ACT;
    constexpr int NTILE_LD = 8;        // loads of 16 bytes a thread and slice
    static_assert(2 * STAGE + NW * STG + (BIASED ? 2 * NW * 256 : 16) <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
    __shared__ __attribute__((aligned(1024))) char stage_smem[NW * STG];
    // The bias of a wave's 128 columns, one slot a wave and tile parity: it comes with the tile's first slice.
    __shared__ __attribute__((aligned(256))) char bias_smem[BIASED ? 2 * NW * 256 : 16];

    // (The lane is formed afresh, lane_now, wherever it is needed: held, with all that follows from it, it would not
    // fit the registers beside the K loop's.)
    const int wid = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wid >> 1, wn = wid & 1;
    const uint32_t smem_lds = (uint32_t)(uintptr_t)(GBA_LDS void *)smem;
    const int N = g.N;
    const uint32_t KB = (uint32_t)g.K * 2u;   // bytes (values) of a row
    const int nk = ceil_div(g.K, 64);         // slices of a tile
    const int tail = KB % 128 ? nk - 1 : -1;
    const int blocks_n = ceil_div(N, 128), tiles_n = ceil_div(N, BN);

    // Up to 64 experts: lane l holds the rows of expert l and the row tiles of experts 0 .. l.
    int upto = 0, row_tiles = 0, start_l = 0, rows_l = 0;
    const bool few = g.E <= 64;
    if (few) {
        const int lane = lane_now();
        if (lane < g.E) gbx::expert_rows(g, lane, start_l, rows_l);
        upto = gbx::wave_scan(ceil_div(rows_l, BM), lane);
        row_tiles = min(__builtin_amdgcn_readlane(upto, 63), g.row_bound);
    } else {
        row_tiles = gbx::total_row_tiles(g, BM, lane_now());
    }
    const int T = row_tiles * tiles_n, G = min((int)gridDim.x, T);
    if ((int)blockIdx.x >= G) return;
    const int slot = xcd_remap(blockIdx.x, G);

    struct Tile {
        int e, start, m0, n0, rows;
    };
    auto tile_of = [&](int r, Tile &t) __attribute__((always_inline)) -> bool {
        const int idx = r * G + slot;
        if (idx >= T) return false;
        const int rt = idx / tiles_n;
        const Found f = few ? gbx::few_row_tile(upto, start_l, rows_l, rt) : gbx::find_row_tile(g, BM, rt, lane_now());
        int tm, tn;
        t.e = f.e;
        t.start = f.start;
        t.rows = f.rows;
        grouped_tile(idx - f.before * tiles_n, f.tiles, tiles_n, 4, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
        return true;
    };

    // ---- loads: a thread's rows tid / 8 + 64 i of each tile, chunk (tid % 8) ^ (row % 8) ----
    uint32_t off[4];
    auto set_off = [&](bool last) __attribute__((always_inline)) {
        const int tid = wid * 64 + lane_now(), chunk = (tid & 7) ^ ((tid >> 3) & 7);
        const bool ok = !last || (uint32_t)(tail * 128 + chunk * 16) < KB;
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = ok ? (uint32_t)((tid >> 3) + 64 * i) * KB + (uint32_t)chunk * 16u : kOobOffset;
    };
    struct Pos {
        const char *pa, *pb;
        const uint32_t *ps, *pw;
        uint32_t na, nb, ns, nw;
    };
    auto pos_full = [&](const Tile &t, bool live, int kt) __attribute__((always_inline)) {
        Pos p;
        const uint32_t k0 = (uint32_t)kt * 128u;
        const int rows_a = min(t.rows - t.m0, BM), rows_b = min(N - t.n0, BN);
        p.pa = (const char *)g.A + ((size_t)(t.start + t.m0) * KB + k0);
        p.na = live ? (uint32_t)rows_a * KB - k0 : 0u;
        p.pb = (const char *)g.B + (((size_t)t.e * N + t.n0) * KB + k0);
        p.nb = live ? (uint32_t)rows_b * KB - k0 : 0u;
        p.ps = g.sa + (size_t)kt * g.T + t.start + t.m0;
        p.ns = live ? (uint32_t)rows_a * 4u : 0u;
        // (The second half of a tile may lie past the last block of columns.)
        p.pw = g.sb + ((size_t)t.e * blocks_n + min(t.n0 / 128 + wn, blocks_n - 1)) * nk + kt;
        p.nw = live ? 4u : 0u;
        return p;
    };
    auto pos_next = [&](Pos &p) __attribute__((always_inline)) {
        p.pa += 128;
        p.na -= 128u;
        p.pb += 128;
        p.nb -= 128u;
        p.ps += g.T;
        p.pw += 1;
    };
    const uint32_t ld_wave = __builtin_amdgcn_readfirstlane(smem_lds + (uint32_t)(wid * 1024));
    // Load i of the slice at p into the stage at byte `st`: 0 - 3 A, 4 - 7 W, 8 A's scales, 9 W's.
    auto dma_one = [&](uint32_t st, const Pos &p, auto i_c) __attribute__((always_inline)) {
        constexpr int i = decltype(i_c)::value;
        if constexpr (i < 4) {
            buffer_load_lds16(make_rsrc(p.pa, p.na), off[i], ld_wave + st + (uint32_t)(i * 8192));
        } else if constexpr (i < 8) {
            buffer_load_lds16(make_rsrc(p.pb, p.nb), off[i - 4], ld_wave + st + (uint32_t)(TILE + (i - 4) * 8192));
        } else if constexpr (i == 8) {
            // 64 rows a wave, by two waves alike.
            buffer_load_lds4(make_rsrc(p.ps, p.ns), (uint32_t)((wid & 3) * 256 + lane_now() * 4), smem_lds + st + (uint32_t)(SCALES + (wid & 3) * 256));
        } else {
            buffer_load_lds4(make_rsrc(p.pw, p.nw), 0u, smem_lds + st + (uint32_t)(SCALES + 1024 + wid * 256));
        }
    };
    constexpr int LD = NTILE_LD + 2;
    auto bias_dma = [&](const Tile &t, int parity) __attribute__((always_inline)) {
        const int cols = min(N - t.n0 - wn * WTN, WTN);
        const uint16_t *const b = g.bias + (size_t)t.e * N + t.n0;
        buffer_load_lds4(make_rsrc(cols > 0 ? b + wn * WTN : b, cols > 0 ? (uint32_t)cols * 2u : 0u), (uint32_t)lane_now() * 4u,
                         (uint32_t)(uintptr_t)(GBA_LDS void *)bias_smem + (uint32_t)((parity * NW + wid) * 256));
    };

    // ---- fragments ----
    // Row 16 f + tj of the wave's rows: 128 bytes, chunk c at c ^ (tj % 8); chunks tg and tg + 4.
    uint32_t a_at, w_at;
    {
        const int tj = lane_now() & 15, tg = lane_now() >> 4;
        const uint32_t at = (uint32_t)(tj * 128 + ((tg ^ (tj & 7)) * 16));
        a_at = smem_lds + (uint32_t)(wm * WTM * 128) + at;
        w_at = smem_lds + (uint32_t)(TILE + wn * WTN * 128) + at;
    }
    auto frag = [&](uint32_t base, int f) __attribute__((always_inline)) {
        const u32x4 x = *(GBA_LDS const u32x4 *)(base + (uint32_t)(f * 2048));
        const u32x4 y = *(GBA_LDS const u32x4 *)((base ^ 64u) + (uint32_t)(f * 2048));
        return gbx::i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
    };
    gbx::i32x8 fa[FM], fw[2][2];
    float sa[FM], sw, s[FM], s_old[FM];   // scales as read; their products, of this slice and the last
    float acc[FN][FM][4];
    f32x4 t[LAG + 1];
    auto read_scales = [&](uint32_t st) __attribute__((always_inline)) {
        const uint32_t lane = (uint32_t)lane_now(), base = smem_lds + st + (uint32_t)SCALES;
#pragma unroll
        for (int f = 0; f < FM; ++f) sa[f] = *(GBA_LDS const float *)(base + (uint32_t)(wm * WTM * 4 + f * 64) + (lane & 15) * 4);
        sw = *(GBA_LDS const float *)(base + (uint32_t)(1024 + wid * 256) + lane * 4);
    };

    Tile cur;
    if (!tile_of(0, cur)) return;
    Pos pos = pos_full(cur, true, 0);
    set_off(false);
    if (BIASED && g.bias) bias_dma(cur, 0);
    static_for<LD>([&](auto i_c) { dma_one(0u, pos, i_c); });
    set_off(tail == 1);
    pos = pos_full(cur, true, 1);
    static_for<4>([&](auto i_c) { dma_one((uint32_t)STAGE, pos, i_c); });
    wait_vmcnt<4>();
    block_barrier();
    uint32_t st = 0;   // this slice's stage, in bytes
    auto read_first = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < FM; ++f) fa[f] = frag(a_at + st, f);
#pragma unroll
        for (int f = 0; f < 2; ++f) fw[0][f] = frag(w_at + st, f);
        read_scales(st);
    };
    read_first();

    // Product q of a slice: column block q / 4, row block q % 4.
    for (int r = 0;; ++r) {
        Tile nxt;
        const bool nxt_live = tile_of(r + 1, nxt);
        if (!nxt_live) nxt = cur;

        auto slice = [&](int kt, auto first_c) __attribute__((always_inline)) {
            constexpr bool FIRST = decltype(first_c)::value;
            const uint32_t other = (uint32_t)STAGE - st;
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                s_old[f] = s[f];
                s[f] = sa[f] * sw;
            }
            // The slice two ahead: this tile's, or the next one's first two.
            const bool here = kt + 2 < nk;
            static_for<4>([&](auto g_c) __attribute__((always_inline)) {
                constexpr int gr = decltype(g_c)::value;
                if constexpr (gr < 3) {
#pragma unroll
                    for (int f = 0; f < 2; ++f) fw[(gr + 1) & 1][f] = frag(w_at + st, 2 * gr + 2 + f);
                    if constexpr (gr == 1) {
                        pos_next(pos);
                        if (__builtin_expect(kt + 3 >= nk, 0)) {
                            const int k2 = here ? kt + 2 : kt + 2 - nk;
                            set_off(k2 == tail);
                            pos = pos_full(here ? cur : nxt, here | nxt_live, k2);
                            if (BIASED && g.bias && !here && k2 == 0 && nxt_live) bias_dma(nxt, (r + 1) & 1);
                        }
                    }
                } else {
                    wait_vmcnt_lgkm0<0>();
                    block_barrier();
                }
                static_for<8>([&](auto q_c) __attribute__((always_inline)) {
                    constexpr int h = decltype(q_c)::value, q = gr * 8 + h, fn = q / FM;
                    constexpr int fm = q % FM;
                    t[q % (LAG + 1)] = gbx::mfma_f8(fw[gr & 1][h / FM], fa[fm]);
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (q >= LAG) {
                        constexpr int p = q - LAG, pn = p / FM, pm = p % FM;
                        scaled_add<FIRST>(acc[pn][pm], t[p % (LAG + 1)], s[pm]);
                    } else if constexpr (!FIRST) {
                        constexpr int p = NMF + q - LAG, pn = p / FM, pm = p % FM;
                        scaled_add<false>(acc[pn][pm], t[p % (LAG + 1)], s_old[pm]);
                    }
                    // (The loads go on in the next slice, whose other stage this one is.)
                    if constexpr (gr == 0 && h < 6) dma_one(other, pos, std::integral_constant<int, 4 + h>{});
                    if constexpr (gr == 3) {
                        if constexpr (h % 2 == 0) dma_one(st, pos, std::integral_constant<int, h / 2>{});
                        if constexpr (h < 2) fw[0][h] = frag(w_at + other, h);
                        if constexpr (h == 2) read_scales(other);
                        if constexpr (h >= 4) fa[fm] = frag(a_at + other, fm);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
            });
            if constexpr (FIRST) {
                // The sums taken up in the next slice start from 0.
#pragma unroll
                for (int p = NMF - LAG; p < NMF; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[p / FM][p % FM][i] = 0.0f;
            }
            st = other;
        };
        slice(0, std::true_type{});
        for (int kt = 1; kt < nk; ++kt) slice(kt, std::false_type{});
        // 32 wait states: more than a matrix instruction needs before its sums are read.
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int p = NMF - LAG; p < NMF; ++p) scaled_add<false>(acc[p / FM][p % FM], t[p % (LAG + 1)], s[p % FM]);

        // ---- epilogue, while the next tile's first slices land ----
        __builtin_amdgcn_sched_barrier(0);
        {
            // 16 rows x 64 columns at a time through a staging buffer, to rows of 128 bytes: chunk c of row r at c ^ (r % 8).
            // (The lane afresh, and the arguments: addresses formed from them ahead of the K loop would not fit the registers.)
            typedef const Group __attribute__((address_space(4))) *ArgPtr;
            ArgPtr ga = (ArgPtr)__builtin_amdgcn_kernarg_segment_ptr();
            asm volatile("" : "+s"(ga));
            const int ln = lane_now(), ej = ln & 15, eg = ln >> 4;   // write side: row, four-column group
            const int rr = ln >> 3, rc = ln & 7;                     // read side: row (of 8), 16-byte chunk
            char *const stg = stage_smem + wid * STG;
            const size_t corner = ((size_t)cur.start + cur.m0 + wm * WTM) * (size_t)N + cur.n0 + wn * WTN;
            const int rows_left = cur.rows - cur.m0 - wm * WTM, cols_left = N - cur.n0 - wn * WTN;
            constexpr bool SLOPED = EPI == gbx::EPI_SLOPE && ACT != ACT_NONE;
            constexpr int A = EPI == gbx::EPI_ACT ? ACT : ACT_NONE;
            const bool with_z = BIASED && ga->zout != nullptr;
            const bool has_bias = BIASED && ga->bias != nullptr;
            // 64 rows of at most 2^24 bytes: offsets below 2^31.
            const __amdgpu_buffer_rsrc_t Cw = make_rsrc((uint16_t *)ga->C + corner, 0x7fffffffu);
            const __amdgpu_buffer_rsrc_t Pw = make_rsrc(with_z ? ga->zout + corner : nullptr, with_z ? 0x7fffffffu : 0u);
            const __amdgpu_buffer_rsrc_t Zw = make_rsrc(SLOPED ? ga->z + corner : nullptr, SLOPED ? 0x7fffffffu : 0u);
            const uint32_t pitch = (uint32_t)N * 2u;
            const uint32_t st_off = (uint32_t)rr * pitch + (uint32_t)rc * 16u, z_off = (uint32_t)ej * pitch + (uint32_t)eg * 8u;
            char *const put = stg + ej * 128 + (eg & 1) * 8;
            const char *const get = stg + rr * 128 + ((rc ^ (rr & 7)) * 16);
            // WHOLE: all 64 x 128 values are there and rows are whole 128-byte lines, which leave non-temporally. (Others
            // share lines with the tile's next stores, and are left to the L2 to join.)
            auto store_all = [&](auto whole_c) __attribute__((always_inline)) {
                constexpr bool WHOLE = decltype(whole_c)::value;
                constexpr int NG = 2 * FM;
                // Group n: rows 16 (n % FM) .., columns 64 (n / FM) ..
                auto send = [&](__amdgpu_buffer_rsrc_t out, const u32x4 (&v)[2], int n) __attribute__((always_inline)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int row = n % FM * 16 + 8 * j, col = n / FM * 64;
                        if constexpr (WHOLE) {
                            __builtin_amdgcn_raw_buffer_store_b128(v[j], out, (int)st_off, (int)((uint32_t)row * pitch) + col * 2, 2 /* nt */);
                        } else {
                            const bool there = row + rr < rows_left && col + rc * 8 < cols_left;
                            __builtin_amdgcn_raw_buffer_store_b128(v[j], out, (int)(there ? st_off + (uint32_t)row * pitch + (uint32_t)col * 2u : kOobOffset), 0, 0);
                        }
                    }
                };
                auto fetch = [&](u32x4 (&v)[2]) __attribute__((always_inline)) {
                    v[0] = *reinterpret_cast<const u32x4 *>(get);
                    v[1] = *reinterpret_cast<const u32x4 *>(get + 1024);
                };
                u32x2 z[2][4];   // of a group (a lane: one row, four columns a block), a group ahead of its use
                auto load_z = [&](int n) __attribute__((always_inline)) {
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const int row = n % FM * 16, col = n / FM * 64 + 16 * f;
                        const bool there = WHOLE || (row + ej < rows_left && col + 4 * eg < cols_left);
                        z[n & 1][f] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(Zw, (int)(there ? z_off + (uint32_t)row * pitch + (uint32_t)col * 2u : kOobOffset), 0, 0));
                    }
                };
                if constexpr (SLOPED) load_z(0);
                f32x4 bq[BIASED ? 4 : 1];
                u32x4 v[2];
#pragma unroll
                for (int n = 0; n <= NG; ++n) {
                    if (n > 0) fetch(v);   // (a wave's LDS instructions run in order)
                    if (n < NG) {
                        const int fm = n % FM, fh = n / FM;
                        if constexpr (SLOPED)
                            if (n + 1 < NG) load_z(n + 1);
                        if constexpr (BIASED) {
                            if (fm == 0) {
#pragma unroll
                                for (int f = 0; f < 4; ++f) {
                                    bq[f] = f32x4{0.f, 0.f, 0.f, 0.f};
                                    if (has_bias) {
                                        const u32x2 b = *reinterpret_cast<const u32x2 *>(bias_smem + ((r & 1) * NW + wid) * 256 + fh * 128 + f * 32 + eg * 8);
                                        bq[f] = f32x4{to_f32<ODT>(b.x & 0xffffu), to_f32<ODT>(b.x >> 16), to_f32<ODT>(b.y & 0xffffu), to_f32<ODT>(b.y >> 16)};
                                    }
                                }
                            }
                        }
                        f32x4 s4[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const float(&q)[4] = acc[4 * fh + f][fm];
                            s4[f] = f32x4{q[0], q[1], q[2], q[3]};
                            if constexpr (BIASED) s4[f] += bq[f];
                        }
                        auto staged = [&](int f) __attribute__((always_inline)) {
                            return reinterpret_cast<u32x2 *>(put + (((2 * f + (eg >> 1)) ^ (ej & 7)) * 16));
                        };
                        if (BIASED && with_z) {
                            u32x4 p[2];
#pragma unroll
                            for (int f = 0; f < 4; ++f) *staged(f) = u32x2{pack2<ODT>(s4[f][0], s4[f][1]), pack2<ODT>(s4[f][2], s4[f][3])};
                            wave_sync();
                            fetch(p);
                            send(Pw, p, n);
                        }
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            f32x4 a = s4[f];
                            if constexpr (SLOPED) {
                                const u32x2 q = z[n & 1][f];
                                a[0] *= gbx::act_slope<ACT>(to_f32<ODT>(q.x & 0xffffu));
                                a[1] *= gbx::act_slope<ACT>(to_f32<ODT>(q.x >> 16));
                                a[2] *= gbx::act_slope<ACT>(to_f32<ODT>(q.y & 0xffffu));
                                a[3] *= gbx::act_slope<ACT>(to_f32<ODT>(q.y >> 16));
                            }
                            *staged(f) = u32x2{pack2<ODT>(act_fn<A>(a[0]), act_fn<A>(a[1])), pack2<ODT>(act_fn<A>(a[2]), act_fn<A>(a[3]))};
                        }
                        wave_sync();
                    }
                    if (n > 0) send(Cw, v, n - 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            if (rows_left >= WTM && cols_left >= WTN && N % 64 == 0)
                store_all(std::true_type{});
            else
                store_all(std::false_type{});
        }
        __builtin_amdgcn_sched_barrier(0);
        if (!nxt_live) break;
        cur = nxt;
        read_first();   // (again: held across the epilogue, the fragments would take its registers)
    }
    wait_vmcnt<0>();   // no direct-to-LDS write may outlive the workgroup's LDS
}

// Grid: one workgroup per CU, or fewer for fewer tiles. Two slices at least (K > 128).
template <int ODT, int EPI, int ACT>
hipError_t launch_f8_persist(Group g, hipStream_t stream) {
    const long long tiles_n = ceil_div(g.N, 256), row_tiles = gbx::row_tile_bound(g.T, g.E, 256), tiles = row_tiles * tiles_n;
    if (tiles <= 0) return hipSuccess;
    // Tile indices r * G + slot run up to tiles + G - 1: keep them in int.
    if (tiles > 0x7fffffffLL - 0x10000 || g.K <= 64) return hipErrorInvalidValue;
    g.row_bound = (int)row_tiles;
    int cus = 0;
    const hipError_t e = current_cus(&cus);
    if (e != hipSuccess) return e;
    return launch(f8_persist_kernel<ODT, EPI, ACT>, dim3((unsigned)(tiles < cus ? tiles : cus)), dim3(512), stream, g);
}

}  // namespace gbm
