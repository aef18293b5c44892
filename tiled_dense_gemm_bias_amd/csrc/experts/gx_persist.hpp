// Persistent kernel of the large grouped products: one workgroup per CU walks
// its 256 x 256 tiles, over all experts, as one stream of 64-word K slices
// through a two-stage LDS ring. The loop is the dense persistent kernel's
// (gemm_v5.hpp, which explains its schedule); what differs:
//
//  * A tile names its expert: the operands' corners, the row edge and (weight
//    gradients) the depth of the sum are the tile's own. The number of tiles is
//    known on the device only: each wave counts the experts' row tiles once (a
//    scan over the lanes, kept in one register for up to 64 experts) and finds a tile's
//    expert with a ballot.
//  * Weight gradients sum over the rows of an expert: a tile has as many slices
//    as its expert's rows fill, and two at least (the stream's prologue), of
//    which those past the rows read nothing and add zeros. An empty expert's tile
//    so comes out as zeros.
//  * 4-bit operands: a slice of 128 bytes a row is 256 codes, and one
//    16 x 16 x 128 scaled matrix instruction takes the place of each 16 x 16 x 32
//    one. A slice's scales (two planes of 256 dwords for each operand, 4 KiB) come
//    with one more load a wave; a lane reads its row's dword and shifts its block's byte down.
//  * Epilogues: bias and activation with the pre-activation beside it, the
//    product with act'(z), gradients in 16 or 32 bits.
//
// What bounds it: the matrix cores at the clock that the power limit leaves (1.9 to
// 2.1 GHz). 16384 rows by 8 even experts of 8192 x 4096 bf16: 728 us, 1.51 PFLOP/s, 74 % of
// the cycles in matrix instructions; with uneven experts 770 (68 row tiles for 64),
// with bias and GELU 842 (8 us of vector arithmetic a tile), with the pre-activations
// 868. 8192 x 14336 x 4096 in 4 bits: 216 us, 4.45 PFLOP/s, 252 with bias and GELU: 16
// slices a tile, of 1.5 us (1.7 GHz), then 7 us of stores and 5 of bias and GELU.
#pragma once

#include "gx_common.hpp"
#include "gemm_v5.hpp"   // lane_now, buffer_load_lds16_at

namespace gbx {

// acc += A.B on one pair of 16-row blocks (16 x 16 x 32, or 16 x 16 x 128 4-bit
// codes with their scales), the accumulator tied to the destination in
// accumulation registers: the compiler's own forms left it free to copy or spill
// accumulators in the K loop once the epilogue grew. It sees neither the
// instruction's latency nor its hazards: the operands come from LDS reads, whose
// waits it places, never straight from vector arithmetic (see shift_scale), and the
// epilogue starts with a gap. FIRST: the sum starts at 0.
template <int OP, bool FIRST>
__device__ __forceinline__ void mfma_tied(f32x4 &acc, const u32x4 &a, const u32x4 &b, uint32_t sa, uint32_t sb) {
    if constexpr (OP == OP_MX4) {
        if constexpr (FIRST)
            asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                         : "=a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
        else
            asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                         : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
    } else if constexpr (OP == OP_F16) {
        if constexpr (FIRST)
            asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, 0" : "=a"(acc) : "v"(a), "v"(b));
        else
            asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    } else {
        if constexpr (FIRST)
            asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, 0" : "=a"(acc) : "v"(a), "v"(b));
        else
            asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    }
}

// 32 wait states: more than a matrix instruction needs between writing an
// accumulator and a vector instruction reading it.
__device__ __forceinline__ void mfma_gap() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// acc += A.B as mfma_tied, with the sums in vector registers (bias gradients).
template <int OP>
__device__ __forceinline__ void mfma_ones(f32x4 &acc, const u32x4 &a, const u32x4 &b) {
    if constexpr (OP == OP_F16)
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(acc) : "v"(a), "v"(b));
    else
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(acc) : "v"(a), "v"(b));
}

// The ACT of an EPI_GRAD kernel names its output, 16 bits or fp32, and whether it
// also sums the columns of dC (the bias gradient), its first factor or its second.
enum { GRAD_16 = 0, GRAD_F32 = 1, GRAD_SUMS_A = 2, GRAD_SUMS_B = 4, kNumGrads = 6 };

template <int OP, int ODT, int EPI, int ACT, bool TB, bool TA>
__global__ void __launch_bounds__(256)
grouped_persist_kernel(Group g) {
    constexpr bool MX = OP == OP_MX4;
    constexpr int BM = 256, BN = 256, BK = 64, BD = 16, KS = 32, KK = 2, WN = 2;
    constexpr int NW = 4, NT = 256, CH = 8, CHW = 32;   // chunks of a K-contiguous row; of a k row
    constexpr int WTM = 128, WTN = 128, FM = 8, FN = 8;
    constexpr int NFA = (TA ? 2 : 1) * FM, NFB = (TB ? 1 : 2) * FN;
    constexpr int NMF = FM * FN, NPF = NFA + NFB + (MX ? FM + FN : 0);
    constexpr int TILE_BYTES = 32768;
    constexpr uint32_t B_REGION = 2 * TILE_BYTES, S_REGION = 4 * TILE_BYTES;   // A's stages, B's, the scales'
    constexpr int S_BYTES = MX ? 4096 : 0;   // a stage's scales: A's two planes, B's two
    constexpr int LD = 16, EVERY = NMF / LD, LDS_LOADS = LD + (MX ? 1 : 0);
    static_assert(!TA || (!TB && !MX), "layouts: nt, nn, tn");
    static_assert(!MX || TB, "4-bit operands are K-contiguous");
    constexpr bool BIASED = EPI == EPI_ACT;
    constexpr bool GRAD = EPI == EPI_GRAD, SUMS_A = GRAD && (ACT & GRAD_SUMS_A) != 0;
    constexpr bool SUMS = SUMS_A || (GRAD && (ACT & GRAD_SUMS_B) != 0);

    __shared__ __attribute__((aligned(1024))) char smem[4 * TILE_BYTES + 2 * S_BYTES];
    // A tile's bias, one 1 KiB slot per wave and per tile parity (see gemm_v5.hpp).
    __shared__ __attribute__((aligned(1024))) char bias_smem[BIASED ? 2 * NW * 1024 : 16];
    constexpr int STG_BYTES = 16 * 64 * 2;
    __shared__ __attribute__((aligned(1024))) char stage_smem[NW * 2 * STG_BYTES];
    // Where the loads that warm the L2 drop what they read (4-bit: no LDS left for it).
    constexpr bool WARM = !MX;
    constexpr int WARM_BY = 3;
    __shared__ __attribute__((aligned(256))) char warm_smem[WARM ? 256 : 16];
    static_assert(4 * TILE_BYTES + 2 * S_BYTES + 2 * NW * 1024 + NW * 2 * STG_BYTES + (WARM ? 256 : 0) <= 160 * 1024, "LDS");

    const int wid_s = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int K = g.K, N = g.N;   // rows mode: the depth; TA: the tile's (nk below)
    const int tail_k = !TA && (K % BK) != 0 ? (K + BK - 1) / BK - 1 : -1;
    const uint32_t smem_lds = (uint32_t)(uintptr_t)(GBA_LDS void *)smem;
    const int tiles_n = ceil_div(N, BN), tiles_m_ta = TA ? ceil_div(g.M, BM) : 0;

    // Up to 64 experts: lane l holds the first row and the rows of expert l, and (rows
    // mode) the row tiles of experts 0 .. l, so that a tile's expert costs no memory access.
    int upto = 0, row_tiles = 0, start_l = 0, rows_l = 0;
    const bool few = g.E <= 64;
    if (few) {
        const int l = lane_now();
        if (l < g.E) expert_rows(g, l, start_l, rows_l);
        if constexpr (!TA) {
            upto = wave_scan(ceil_div(rows_l, BM), l);
            row_tiles = min(__builtin_amdgcn_readlane(upto, 63), g.row_bound);
        }
    } else if constexpr (!TA) {
        row_tiles = total_row_tiles(g, BM, lane_now());
    }
    const int T = TA ? g.E * tiles_m_ta * tiles_n : row_tiles * tiles_n;
    const int G = min((int)gridDim.x, T);
    if ((int)blockIdx.x >= G) return;
    const int slot = xcd_remap(blockIdx.x, G);

    struct Tile {
        int e, start, m0, n0, rows;   // rows: of the expert's output (TA: all M)
        int klen, nk;                 // depth of the sum, slices streamed
    };
    auto tile_of = [&](int r, Tile &t) -> bool {
        const int idx = r * G + slot;
        if (idx >= T) return false;
        int tm, tn;
        if constexpr (TA) {
            t.e = idx / (tiles_m_ta * tiles_n);
            grouped_tile(idx - t.e * tiles_m_ta * tiles_n, tiles_m_ta, tiles_n, 4, tm, tn);
            if (few) {
                t.start = __builtin_amdgcn_readlane(start_l, t.e);
                t.klen = __builtin_amdgcn_readlane(rows_l, t.e);
            } else {
                expert_rows_uniform(g, t.e, t.start, t.klen);
            }
            t.rows = g.M;
            t.nk = max(ceil_div(t.klen, BK), 2);
        } else {
            const int rt = idx / tiles_n;
            const Found f = few ? few_row_tile(upto, start_l, rows_l, rt) : find_row_tile(g, BM, rt, lane_now());
            t.e = f.e;
            t.start = f.start;
            t.rows = f.rows;
            grouped_tile(idx - f.before * tiles_n, f.tiles, tiles_n, 4, tm, tn);
            t.klen = K;
            t.nk = ceil_div(K, BK);
        }
        t.m0 = tm * BM;
        t.n0 = tn * BN;
        return true;
    };

    // ---- loads (offsets and masks as in gemm_v5.hpp) ----
    uint32_t av[8], bv[8], tv[8];
    auto set_av = [&](bool tail) __attribute__((always_inline)) {
        const int t = wid_s * 64 + lane_now();
        const int ca = (t & 7) ^ ((t >> 3) & 7);
        const bool ok = !tail || tail_k * BK + ca * 8 < K;
        const uint32_t base = (uint32_t)(t >> 3) * (uint32_t)K * 2u + (uint32_t)ca * 16u;
#pragma unroll
        for (int i = 0; i < 8; ++i) av[i] = ok ? base + (uint32_t)(i * 64) * (uint32_t)K : kOobOffset;
    };
    auto set_wide = [&](uint32_t (&v)[8], int x0, int pitch) __attribute__((always_inline)) {
        const int t = wid_s * 64 + lane_now();
        const int cb0 = (t & 31) ^ bswz<CHW>(t >> 5);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = cb0 ^ (8 * (j & 3));
            v[j] = x0 + c * 8 < pitch ? (uint32_t)((t >> 5) + 8 * j) * (uint32_t)pitch * 2u + (uint32_t)c * 16u
                                      : kOobOffset;
        }
    };
    struct SliceDma {
        __amdgpu_buffer_rsrc_t ra, rb, rs;
    };
    struct DmaPos {
        const uint16_t *pa, *pb;
        uint32_t na, nb;
        const uint32_t *ps;   // MX4: this wave's plane of scales
        uint32_t ns;
    };
    // MX4: waves 0, 1 load A's planes, waves 2, 3 B's; dwords between planes.
    const size_t plane_dwords = MX ? (wid_s < 2 ? (size_t)g.T : (size_t)g.E * N) : 0;
    auto pos_full = [&](const Tile &t, bool live, int kt) __attribute__((always_inline)) {
        const int k0 = kt * BK;
        // (readfirstlane: the compiler makes this clamp a vector instruction)
        const uint32_t kin = __builtin_amdgcn_readfirstlane(live && k0 < t.klen ? (uint32_t)min(t.klen - k0, BK) : 0u);
        DmaPos p;
        if constexpr (TA) {
            p.pa = g.A + ((size_t)(t.start + (kin ? k0 : 0)) * g.M + t.m0);
            p.na = kin * (uint32_t)g.M * 2u;
            p.pb = g.B + ((size_t)(t.start + (kin ? k0 : 0)) * N + t.n0);
            p.nb = kin * (uint32_t)N * 2u;
        } else {
            p.pa = g.A + ((size_t)(t.start + t.m0) * K + k0);
            p.na = live ? (uint32_t)min(t.rows - t.m0, BM) * (uint32_t)K * 2u - (uint32_t)k0 * 2u : 0u;
            const uint16_t *const we = g.B + (size_t)t.e * K * N;
            if constexpr (TB) {
                p.pb = we + ((size_t)t.n0 * K + k0);
                p.nb = live ? (uint32_t)min(N - t.n0, BN) * (uint32_t)K * 2u - (uint32_t)k0 * 2u : 0u;
            } else {
                p.pb = we + ((size_t)k0 * N + t.n0);
                p.nb = kin * (uint32_t)N * 2u;
            }
        }
        if constexpr (MX) {
            const int plane = 2 * kt + (wid_s & 1);
            const bool there = live && plane * 32 < K;
            p.ps = (wid_s < 2 ? g.sa + (size_t)t.start + t.m0 : g.sb + (size_t)t.e * N + t.n0) +
                   (there ? (size_t)plane * plane_dwords : 0);
            p.ns = there ? (uint32_t)(wid_s < 2 ? min(t.rows - t.m0, BM) : min(N - t.n0, BN)) * 4u : 0u;
        }
        return p;
    };
    auto pos_next = [&](DmaPos &p) __attribute__((always_inline)) {
        if constexpr (TA) {
            p.pa += (size_t)BK * g.M;
        } else {
            p.pa += BK;
            p.na -= 2u * BK;
        }
        if constexpr (TB) {
            p.pb += BK;
            p.nb -= 2u * BK;
        } else {
            p.pb += (size_t)BK * N;
        }
        if constexpr (MX) p.ps += 2 * plane_dwords;
    };
    auto pin = [](DmaPos &p) __attribute__((always_inline)) {
        asm volatile("" : "+s"(p.pa), "+s"(p.pb), "+s"(p.na), "+s"(p.nb));
        if constexpr (MX) asm volatile("" : "+s"(p.ps), "+s"(p.ns));
    };
    auto make_dma = [](const DmaPos &p) __attribute__((always_inline)) {
        SliceDma d;
        d.ra = make_rsrc(p.pa, p.na);
        d.rb = make_rsrc(p.pb, p.nb);
        if constexpr (MX) d.rs = make_rsrc(p.ps, p.ns);
        return d;
    };
    const uint32_t ld_wave = __builtin_amdgcn_readfirstlane(smem_lds + (uint32_t)(wid_s * 64 * 16));
    // Load i of slice d into the stage whose A region starts (for this wave) at lds_stage; load 16: scales,
    // 1 KiB of the stage's 4 a wave.
    auto dma_one = [&](uint32_t lds_stage, const SliceDma &d, auto i_c) __attribute__((always_inline)) {
        constexpr int i = decltype(i_c)::value;
        if constexpr (i < 8) {
            buffer_load_lds16_at<(uint32_t)(i * NT * 16)>(d.ra, TA ? tv[i] : av[i], lds_stage);
        } else if constexpr (i < 16) {
            buffer_load_lds16_at<B_REGION + (uint32_t)((i - 8) * NT * 16)>(d.rb, TB ? av[i - 8] : bv[i - 8], lds_stage);
        } else {
            // stage byte offset from the first stage is 0 or 32 KiB; the scales' stages are 4 KiB apart
            const uint32_t st = (lds_stage - ld_wave) >> 3;
            buffer_load_lds16_at<S_REGION>(d.rs, (uint32_t)lane_now() * 16u, ld_wave + st);
        }
    };
    // One load a wave and slice warms the L2 for the slice WARM_BY after the one whose loads
    // have just gone out, one lane a 128-byte line: waves 0 and 1 a quarter of B's slice,
    // waves 2 and 3 a quarter of A's; the tiles next to this one, at work on the same
    // XCD, take the other quarters. What it reads lands in LDS that nothing reads. A
    // slice's own loads have half a slice to a whole one (0.6 to 1.2 us) to arrive, too
    // little for HBM, where a round's rows and weights come from when each expert has
    // its own: 16384 x 8192 x 4096 bf16 by 8 experts 793 -> 751 us (one expert, whose
    // weights the caches hold, 715 -> 720), weight gradients 835 -> 786. By two slices instead
    // of three the same within 1 %, of B alone nothing, every line by its own tile 2 % less gain.
    const uint32_t warm_lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(GBA_LDS void *)warm_smem);
    const bool warm_b = wid_s < 2;
    uint32_t warm_off = 0;   // this lane's line, from the slice's corner
    auto set_warm = [&](const Tile &t) __attribute__((always_inline)) {
        const bool wide = warm_b ? !TB : TA;
        const uint32_t pitch = (uint32_t)(warm_b ? (TB ? K : N) : (TA ? g.M : K)) * 2u;
        const int quarter = ((warm_b ? t.m0 : t.n0) >> 8) & 3, l = lane_now(), w = wid_s & 1;
        warm_off = l >= 32 ? kOobOffset
                   : wide  ? (uint32_t)(quarter * 16 + w * 8 + (l >> 2)) * pitch + (uint32_t)(l & 3) * 128u
                           : (uint32_t)(quarter * 64 + w * 32 + l) * pitch;
        asm volatile("" : "+v"(warm_off));
    };
    // Position and range of the slice WARM_BY after the one at p (`there`: not past the tile's last whole one).
    auto warm_at = [&](const DmaPos &p) __attribute__((always_inline)) {
        const uint16_t *const a = TA ? p.pa + (size_t)(WARM_BY * BK) * g.M : p.pa + WARM_BY * BK;
        const uint16_t *const b = TB ? p.pb + WARM_BY * BK : p.pb + (size_t)(WARM_BY * BK) * N;
        return warm_b ? b : a;
    };
    auto warm_bytes = [&](const DmaPos &p, bool there) __attribute__((always_inline)) {
        const uint32_t n = warm_b ? p.nb - (TB ? 2u * WARM_BY * BK : 0u) : p.na - (TA ? 0u : 2u * WARM_BY * BK);
        return there ? n : 0u;
    };
    auto warm = [&](__amdgpu_buffer_rsrc_t rs) __attribute__((always_inline)) {
        asm volatile(
            "s_mov_b32 m0, %2\n\t"
            "s_nop 0\n\t"
            "buffer_load_dword %0, %1, 0 offen lds"
            :
            : "v"(warm_off), "s"(rs), "s"(warm_lds)
            : "memory", "m0");
    };
    const uint32_t bias_lds = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(GBA_LDS void *)bias_smem + (uint32_t)(wid_s * 1024));
    auto bias_dma = [&](const Tile &t, int p) {
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(g.bias + (size_t)t.e * N + t.n0, (uint32_t)min(N - t.n0, BN) * 2u);
        const int l = lane_now();
        buffer_load_lds16(rb, l < BN / 8 ? (uint32_t)l * 16u : kOobOffset, bias_lds + (uint32_t)(p * NW * 1024));
    };

    // ---- fragments (bases as in gemm_v5.hpp) ----
    constexpr int NBB = TB ? KK : FN, NBA = TA ? FM : KK;
    uint32_t fa_base[TA ? 1 : KK], fb_base[NBB], ft_base[TA ? FM : 1];
    uint32_t sc_base[MX ? 2 : 1];   // MX4: this lane's scale dwords of A's and B's first blocks, kk = 0
    auto set_bases = [&](uint32_t st) __attribute__((always_inline)) {
        const int l = lane_now();
        const int tg = l >> 4, tj = l & 15;
        const int wm_s = wid_s / WN, wn_s = wid_s % WN;
        const uint32_t s0 = smem_lds + st;
        if constexpr (!TA) {
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const int r = wm_s * WTM + tj;
                fa_base[kk] = s0 + (uint32_t)(r * (BK * 2) + aswz<16, CH>(r, (KS / 8) * kk + tg) * 16);
            }
        }
#pragma unroll
        for (int f = 0; f < NBB; ++f) {
            if constexpr (TB) {
                const int r = wn_s * WTN + tj;
                fb_base[f] = s0 + B_REGION + (uint32_t)(r * (BK * 2) + aswz<16, CH>(r, (KS / 8) * f + tg) * 16);
            } else {
                const int k = 8 * tg + (tj >> 2);
                const int n = wn_s * WTN + f * 16 + 4 * (tj & 3);
                const int c = (n >> 3) ^ bswz<CHW>(k);
                fb_base[f] = s0 + B_REGION + (uint32_t)(k * (BN * 2) + c * 16 + (n & 4) * 2);
            }
        }
        if constexpr (TA) {
            const int k = 8 * tg + (tj >> 2);
            const int m = wm_s * WTM + 4 * (tj & 3);
            const int c = (m >> 3) ^ bswz<CHW>(k);
            const uint32_t b0 = (uint32_t)(k * (BM * 2) + c * 16 + (m & 4) * 2);
#pragma unroll
            for (int fm = 0; fm < FM; ++fm) ft_base[fm] = s0 + (b0 ^ (uint32_t)(fm << 5));
        }
        if constexpr (MX) {
            sc_base[0] = smem_lds + S_REGION + (st >> 3) + (uint32_t)((wm_s * WTM + tj) * 4);
            sc_base[1] = smem_lds + S_REGION + (st >> 3) + (uint32_t)(2048 + (wn_s * WTN + tj) * 4);
        }
    };
    set_bases(0u);

    f32x4 acc[FN][FM];
    u32x4 fa[2][FM];
    i16x4 fal[2][FM], fah[2][FM];
    i16x4 fbl[2][FN], fbh[2][FN];
    u32x4 fw[2][FN];
    uint32_t sca[2][FM], scb[2][FN];
    // The column sums of dC, as products with ones: one more matrix instruction for each of
    // dC's fragments, in the tiles of the other factor's first 256 columns and the
    // waves of its first 128. A pass of its own over dC took 54 us beside 744 (16384 rows,
    // 8 experts of 8192 x 4096), these 21; kernels of their own, as the branch alone costs 20.
    f32x4 sums[SUMS ? FM : 1];
    constexpr uint32_t kOne = OP == OP_F16 ? 0x3c003c00u : 0x3f803f80u;
    u32x4 ones = {kOne, kOne, kOne, kOne};
    if constexpr (SUMS) asm volatile("" : "+v"(ones));
    auto add_sums = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            if constexpr (SUMS_A)
                mfma_ones<OP>(sums[f], ones, __builtin_bit_cast(u32x4, __builtin_shufflevector(fal[buf][f], fah[buf][f], 0, 1, 2, 3, 4, 5, 6, 7)));
            else
                mfma_ones<OP>(sums[f], __builtin_bit_cast(u32x4, __builtin_shufflevector(fbl[buf][f], fbh[buf][f], 0, 1, 2, 3, 4, 5, 6, 7)), ones);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto read_one = [&](int buf, int kk, int r) __attribute__((always_inline)) {
        if (r < NFA) {
            if constexpr (TA) {
                const int fm = r >> 1, h = r & 1;
                const uint32_t o = (uint32_t)((32 * kk + 4 * h) * (BM * 2));
                const i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GBA_LDS i16x4 *)(ft_base[fm] + o));
                if (h)
                    fah[buf][fm] = v;
                else
                    fal[buf][fm] = v;
            } else {
                fa[buf][r] = *(GBA_LDS const u32x4 *)(fa_base[kk] + (uint32_t)(r * BD * (BK * 2)));
            }
        } else if (r < NFA + NFB) {
            if constexpr (TB) {
                const int fn = r - NFA;
                fw[buf][fn] = *(GBA_LDS const u32x4 *)(fb_base[kk] + (uint32_t)(fn * BD * (BK * 2)));
            } else {
                const int fn = (r - NFA) >> 1, h = (r - NFA) & 1;
                const uint32_t o = (uint32_t)((32 * kk + 4 * h) * (BN * 2));
                const i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GBA_LDS i16x4 *)(fb_base[fn] + o));
                if (h)
                    fbh[buf][fn] = v;
                else
                    fbl[buf][fn] = v;
            }
        } else if constexpr (MX) {
            const int f = r - NFA - NFB;
            if (f < FM)
                sca[buf][f] = *(GBA_LDS const uint32_t *)(sc_base[0] + (uint32_t)(kk * 1024 + f * 64));
            else
                scb[buf][f - FM] = *(GBA_LDS const uint32_t *)(sc_base[1] + (uint32_t)(kk * 1024 + (f - FM) * 64));
        }
    };
    // MX4: a row's scale dword has its four blocks' bytes; lane l's is block l / 16.
    // Shifted where no memory instruction is issued, at least two matrix
    // instructions before the first that takes them (the hardware wants two
    // instructions between a vector write and a matrix instruction's read).
    const uint32_t sc_shift = MX ? (uint32_t)(8 * (lane_now() >> 4)) : 0u;
    auto shift_scale = [&](int buf, int f) __attribute__((always_inline)) {
        uint32_t &s = f < FM ? sca[buf][f] : scb[buf][f - FM];
        asm volatile("v_lshrrev_b32 %0, %1, %0" : "+v"(s) : "v"(sc_shift));
    };
    constexpr int SHIFT_Q = NMF - 2 - FM - FN;   // MX4: first MFMA that a shift follows
    static_assert(!MX || SHIFT_Q >= NPF, "scales are read before they are shifted");
    constexpr int NBASE = NBA + NBB + (MX ? 2 : 0);
    static_assert(NPF + NBASE <= NMF, "base moves after the step's reads");
    auto add_to = [](uint32_t &x, int delta) __attribute__((always_inline)) {
        asm volatile("v_add_u32 %0, %1, %0" : "+v"(x) : "s"(delta));
    };
    auto move_base = [&](int b, int delta) __attribute__((always_inline)) {
        if (b < NBA) {
            if constexpr (TA)
                add_to(ft_base[b], delta);
            else
                add_to(fa_base[b], delta);
        } else if (b < NBA + NBB) {
            add_to(fb_base[b - NBA], delta);
        } else {
            add_to(sc_base[b - NBA - NBB], delta >> 3);   // +-4 KiB
        }
    };
    constexpr int PQ = NPF + NBASE + 2;
    static_assert(PQ + 8 < NMF, "payload slots inside the step");
    // (As gemm_v5.hpp's step.)
    auto step = [&](int cur, int pf_kk, auto move_c, int delta, auto dma_c, uint32_t lds_stage,
                    const SliceDma &d, auto first_c, auto &&payload) __attribute__((always_inline)) {
        constexpr bool MOVE = decltype(move_c)::value, DMA = decltype(dma_c)::value;
        constexpr bool FIRST = decltype(first_c)::value;
        static_for<NMF>([&](auto q_c) __attribute__((always_inline)) {
            constexpr int q = decltype(q_c)::value;
            constexpr int fn = q / FM, fm = (fn & 1) ? FM - 1 - q % FM : q % FM;
            u32x4 bop, aop;
            if constexpr (TB)
                bop = fw[cur][fn];
            else
                bop = __builtin_bit_cast(u32x4, __builtin_shufflevector(fbl[cur][fn], fbh[cur][fn], 0, 1, 2, 3, 4, 5, 6, 7));
            if constexpr (TA)
                aop = __builtin_bit_cast(u32x4, __builtin_shufflevector(fal[cur][fm], fah[cur][fm], 0, 1, 2, 3, 4, 5, 6, 7));
            else
                aop = fa[cur][fm];
            mfma_tied<OP, FIRST>(acc[fn][fm], bop, aop, MX ? scb[cur][fn] : 0u, MX ? sca[cur][fm] : 0u);
            if constexpr (q < NPF) read_one(cur ^ 1, pf_kk, q);
            if constexpr (MX && q >= SHIFT_Q && q < SHIFT_Q + FM + FN) shift_scale(cur ^ 1, q - SHIFT_Q);
            if constexpr (MOVE && q >= NPF && q < NPF + NBASE) move_base(q - NPF, delta);
            if constexpr (DMA && q % EVERY == 0) dma_one(lds_stage, d, std::integral_constant<int, q / EVERY>{});
            if constexpr (DMA && MX && q == NMF - 1) dma_one(lds_stage, d, std::integral_constant<int, LD>{});
            payload(q_c);
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    Tile cur_t;
    if (!tile_of(0, cur_t)) return;

    auto set_offsets = [&](const Tile &t, int k) __attribute__((always_inline)) {
        if constexpr (!TA) set_av(k == tail_k);
        if constexpr (!TB) set_wide(bv, t.n0, N);
        if constexpr (TA) set_wide(tv, t.m0, g.M);
    };

    DmaPos pos;
    {
        set_offsets(cur_t, 0);
        if (BIASED && g.bias) bias_dma(cur_t, 0);
        const SliceDma d0 = make_dma(pos_full(cur_t, true, 0));
        static_for<LDS_LOADS>([&](auto i_c) { dma_one(ld_wave, d0, i_c); });
        if (tail_k == 1) set_av(true);
        pos = pos_full(cur_t, true, 1);
        const SliceDma d1 = make_dma(pos);
        static_for<LDS_LOADS>([&](auto i_c) { dma_one(ld_wave + (uint32_t)TILE_BYTES, d1, i_c); });
        if constexpr (WARM) {
            set_warm(cur_t);
            warm(make_rsrc(warm_at(pos), warm_bytes(pos, 2 + WARM_BY < cur_t.nk)));
        }
    }
    wait_vmcnt<LDS_LOADS + (WARM ? 1 : 0)>();
    block_barrier();
    auto read_first = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < NPF; ++q) read_one(0, 0, q);
        if constexpr (MX) {
#pragma unroll
            for (int f = 0; f < FM + FN; ++f) shift_scale(0, f);
            asm volatile("s_nop 1" ::: "memory");   // the wait states of shift_scale
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    read_first();

    uint32_t lds_cur = ld_wave;
    int delta = TILE_BYTES;
    for (int r = 0;; ++r) {
        Tile nxt_t;
        const bool nxt_live = tile_of(r + 1, nxt_t);
        if (!nxt_live) nxt_t = cur_t;
        if (r > 0) {
            set_offsets(cur_t, 1);
            if constexpr (WARM) set_warm(cur_t);
        }
        const int nk = cur_t.nk;
        // The wave that sums: of the tile in the other factor's first columns, the first of two.
        const bool with_sums = SUMS && (SUMS_A ? cur_t.n0 == 0 && wid_s % WN == 0 : cur_t.m0 == 0 && wid_s / WN == 0);
        if constexpr (SUMS) {
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                sums[f] = f32x4{0.f, 0.f, 0.f, 0.f};
                asm volatile("" : "+v"(sums[f]));
            }
        }

        auto slice = [&](int kt, auto first_c) __attribute__((always_inline)) {
            const bool here = kt + 2 < nk;
            const int k2 = here ? kt + 2 : kt + 2 - nk;
            const int k1 = kt + 1 < nk ? kt + 1 : kt + 1 - nk;
            SliceDma dn;
            bool bias_next = false;
            auto prep = [&](auto q_c) __attribute__((always_inline)) {
                constexpr int q = decltype(q_c)::value;
                if constexpr (q == PQ) {
                    pos_next(pos);
                    pin(pos);
                } else if constexpr (q == PQ + 4) {
                    // Near a tile's end (position kt+2 is the tile's last slice, one of the
                    // next tile's first, or past the last tile): offsets and
                    // position from scratch, in one rarely taken block.
                    if (__builtin_expect(kt + 3 >= nk, 0)) {
                        if ((!here) & (k2 == 0) & nxt_live) {
                            if constexpr (!TB) set_wide(bv, nxt_t.n0, N);
                            if constexpr (TA) set_wide(tv, nxt_t.m0, g.M);
                        }
                        if constexpr (!TA)
                            if ((k2 == tail_k) != (k1 == tail_k)) set_av(k2 == tail_k);
                        pos = pos_full(here ? cur_t : nxt_t, here | nxt_live, k2);
                        bias_next = BIASED & (g.bias != nullptr) & (!here) & (k2 == 0) & nxt_live;
                    }
                    pin(pos);
                } else if constexpr (q == PQ + 8) {
                    dn = make_dma(pos);
                    asm volatile("" : "+s"(dn.ra), "+s"(dn.rb));
                    if constexpr (MX) asm volatile("" : "+s"(dn.rs));
                }
            };
            step(0, 1, std::true_type{}, delta, std::false_type{}, 0u, SliceDma{}, first_c, prep);
            if constexpr (SUMS)
                if (with_sums) add_sums(0);
            wait_vmcnt_lgkm0<WARM ? 1 : 0>();   // all but the newest: the load that warms
            block_barrier();
            if (__builtin_expect(bias_next, 0)) bias_dma(nxt_t, (r + 1) & 1);
            __builtin_amdgcn_sched_barrier(0);
            const uint16_t *warm_p = nullptr;
            uint32_t warm_n = 0;
            __amdgpu_buffer_rsrc_t warm_rs = dn.rb;
            step(1, 0, std::false_type{}, 0, std::true_type{}, lds_cur, dn, std::false_type{}, [&](auto q_c) __attribute__((always_inline)) {
                // In pieces, beside matrix instructions that have no other company.
                constexpr int q = decltype(q_c)::value;
                if constexpr (WARM && q == NMF - 11) {
                    warm_p = warm_at(pos);
                    asm volatile("" : "+s"(warm_p));
                } else if constexpr (WARM && q == NMF - 9) {
                    warm_n = warm_bytes(pos, kt + 3 + WARM_BY < nk);
                    asm volatile("" : "+s"(warm_n));
                } else if constexpr (WARM && q == NMF - 6) {
                    warm_rs = make_rsrc(warm_p, warm_n);
                    asm volatile("" : "+s"(warm_rs));
                } else if constexpr (WARM && q == NMF - 1) {
                    warm(warm_rs);
                }
            });
            if constexpr (SUMS)
                if (with_sums) add_sums(1);
            lds_cur += (uint32_t)delta;
            delta = -delta;
        };
        slice(0, std::true_type{});
        for (int kt = 1; kt < nk; ++kt) slice(kt, std::false_type{});
        mfma_gap();

        // ---- epilogue, while the next tile's first slices land ----
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        {
            // The epilogue's arguments, read afresh: held across the K loop they
            // would push other scalars out of their registers.
            typedef const Group __attribute__((address_space(4))) *ArgPtr;
            ArgPtr ga = (ArgPtr)__builtin_amdgcn_kernarg_segment_ptr();
            asm volatile("" : "+s"(ga));
            const bool has_bias = ga->bias != nullptr;
            const int ln = lane_now();
            const int wn_s = wid_s % WN, wm_s = wid_s / WN;
            char *const bias_mine = bias_smem + ((r & 1) * NW + wid_s) * 1024;
            if constexpr (BIASED) {
                if (has_bias) {
                    const uint32_t bb = *reinterpret_cast<const uint32_t *>(bias_mine + wn_s * (WTN * 2) + 4 * ln);
                    *reinterpret_cast<f32x2 *>(bias_mine + 512 + 8 * ln) = f32x2{to_f32<ODT>(bb & 0xffffu), to_f32<ODT>(bb >> 16)};
                }
            }
            char *const stg = stage_smem + wid_s * 2 * STG_BYTES;
            const int wr = ln & 15, wg = ln >> 4;   // write side: row, 4-column group
            const int rr = ln >> 3, rc = ln & 7;    // read side: row (of 8), 16-byte chunk
            // This wave's corner of the output, in values.
            const size_t corner = ((TA ? (size_t)cur_t.e * ga->M : (size_t)cur_t.start) + cur_t.m0 + wm_s * WTM) * (size_t)N +
                                  cur_t.n0 + wn_s * WTN;
            uint32_t st_off = (uint32_t)rr * (uint32_t)N * 2u + (uint32_t)rc * 16u;
            uint32_t pitch8 = __builtin_amdgcn_readfirstlane((uint32_t)N * 16u);
            uint32_t z_off = (uint32_t)wr * (uint32_t)N * 2u + (uint32_t)wg * 8u;   // this lane's place in a block
            asm volatile("" : "+v"(st_off), "+v"(z_off), "+s"(pitch8));
            const int rows_left = cur_t.rows - cur_t.m0 - wm_s * WTM, cols_left = N - cur_t.n0 - wn_s * WTN;
            const bool full = rows_left >= WTM && cols_left >= WTN;
            auto value = [&](int fn, int fm) __attribute__((always_inline)) -> f32x4 {
                f32x4 v;   // the compiler copies it out of its accumulation registers
                asm volatile("" : "=v"(v) : "0"(acc[fn][fm]));
                return v;
            };
            // Rows of whole 128-byte lines leave non-temporally; others share lines with
            // the tile's next stores, and are left to the L2 to join (a weight
            // gradient of 504 columns: 38 us non-temporally).
            const bool lines = N % 64 == 0;
            // (Buffer stores: the compiler joins a non-temporal and an ordinary store of
            // the same value into an ordinary one, and the outputs then push the inputs
            // out of the cache behind the L2: 16384 x 8192 x 4096 711 -> 769 us.)
            auto store16 = [&](__amdgpu_buffer_rsrc_t out, uint32_t at, const u32x4 &v) __attribute__((always_inline)) {
                if (lines)
                    __builtin_amdgcn_raw_buffer_store_b128(v, out, (int)at, 0, 2 /* nt */);
                else
                    __builtin_amdgcn_raw_buffer_store_b128(v, out, (int)at, 0, 0);
            };
            constexpr int NG = 2 * FM;
            // The wave's block through two alternating 16 x 64 staging buffers to
            // rows of 128 bytes (see gemm_v5.hpp). A: activation applied; SLOPED: times act'(z).
            auto store_all = [&](auto masked_c, auto a_c) __attribute__((always_inline)) {
                constexpr bool masked = decltype(masked_c)::value;
                constexpr int A = decltype(a_c)::value;
                constexpr int ZB = 2;
                constexpr bool SLOPED = EPI == EPI_SLOPE && ACT != ACT_NONE;
                // 128 rows of at most 2^24 bytes: offsets below 2^31.
                const __amdgpu_buffer_rsrc_t Cw = make_rsrc((uint16_t *)ga->C + corner, 0x7fffffffu);
                const bool with_z = BIASED && !MX && ga->zout != nullptr;
                const __amdgpu_buffer_rsrc_t Pw = make_rsrc(with_z ? ga->zout + corner : nullptr, with_z ? 0x7fffffffu : 0u);
                f32x4 bq[BIASED ? FN : 1];
                if constexpr (BIASED) {
#pragma unroll
                    for (int f = 0; f < FN; ++f)
                        bq[f] = has_bias ? *reinterpret_cast<const f32x4 *>(bias_mine + 512 + (16 * f + 4 * wg) * 4)
                                         : f32x4{0.f, 0.f, 0.f, 0.f};
                }
                u32x2 zq[SLOPED ? 2 : 1][SLOPED ? ZB : 1][4];
                // z of ZB groups (a lane: one row, four columns), a batch ahead of its use.
                auto load_z = [&](int batch) __attribute__((always_inline)) {
                    const char *const Zw = reinterpret_cast<const char *>(ga->z + corner);
#pragma unroll
                    for (int b = 0; b < ZB; ++b)
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const int fh = (batch * ZB + b) & 1, fm = (batch * ZB + b) >> 1;
                            const uint32_t zo = z_off + (uint32_t)fm * 2u * pitch8 + (uint32_t)(fh * 128 + f * 32);
                            zq[batch & 1][b][f] = !masked || (fm * BD + wr < rows_left && fh * 64 + 16 * f + 4 * wg < cols_left)
                                                      ? *reinterpret_cast<const u32x2 *>(Zw + zo)
                                                      : u32x2{0u, 0u};
                        }
                };
#pragma unroll
                for (int gi = 0; gi <= NG; ++gi) {
                    u32x4 v[2];
                    if (gi > 0) {
                        const char *const sb = stg + ((gi - 1) & 1) * STG_BYTES;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            v[j] = *reinterpret_cast<const u32x4 *>(sb + (8 * j + rr) * 128 + ((rc ^ (rr & 7)) * 16));
                    }
                    if (gi < NG) {
                        const int fh = gi & 1, fm = gi >> 1;
                        char *const sb = stg + (gi & 1) * STG_BYTES;
                        if constexpr (SLOPED) {
                            if (gi == 0) load_z(0);
                            if (gi % ZB == 0 && gi + ZB < NG) load_z(gi / ZB + 1);
                        }
                        f32x4 s[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            s[f] = value(4 * fh + f, fm);
                            if constexpr (BIASED) s[f] += bq[4 * fh + f];
                        }
                        // This lane's 8 bytes of block f, in the staging buffer.
                        auto staged = [&](int f) __attribute__((always_inline)) {
                            const int chunk = 2 * f + (wg >> 1);
                            return reinterpret_cast<u32x2 *>(sb + wr * 128 + ((chunk ^ (wr & 7)) * 16) + (wg & 1) * 8);
                        };
                        if constexpr (BIASED && !MX) {
                            // The pre-activation goes through the same buffer first (a wave's
                            // LDS instructions run in order).
                            if (with_z) {
#pragma unroll
                                for (int f = 0; f < 4; ++f)
                                    *staged(f) = u32x2{pack2<ODT>(s[f][0], s[f][1]), pack2<ODT>(s[f][2], s[f][3])};
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const u32x4 z = *reinterpret_cast<const u32x4 *>(sb + (8 * j + rr) * 128 + ((rc ^ (rr & 7)) * 16));
                                    if (masked && (fm * BD + 8 * j + rr >= rows_left || fh * 64 + rc * 8 >= cols_left)) continue;
                                    const uint32_t offs = st_off + (uint32_t)(2 * fm + j) * pitch8 + (uint32_t)(fh * 128);
                                    store16(Pw, offs, z);
                                }
                            }
                        }
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            f32x4 a = s[f];
                            if constexpr (SLOPED) {
                                const u32x2 z = zq[gi / ZB & 1][gi % ZB][f];
                                a[0] *= act_slope<ACT>(to_f32<ODT>(z.x & 0xffffu));
                                a[1] *= act_slope<ACT>(to_f32<ODT>(z.x >> 16));
                                a[2] *= act_slope<ACT>(to_f32<ODT>(z.y & 0xffffu));
                                a[3] *= act_slope<ACT>(to_f32<ODT>(z.y >> 16));
                            }
                            u32x2 o;
                            o.x = pack2<ODT>(act_fn<A>(a[0]), act_fn<A>(a[1]));
                            o.y = pack2<ODT>(act_fn<A>(a[2]), act_fn<A>(a[3]));
                            *staged(f) = o;
                        }
                    }
                    if (gi > 0) {
                        const int fh = (gi - 1) & 1, fm = (gi - 1) >> 1;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (masked && (fm * BD + 8 * j + rr >= rows_left || fh * 64 + rc * 8 >= cols_left)) continue;
                            const uint32_t offs = st_off + (uint32_t)(2 * fm + j) * pitch8 + (uint32_t)(fh * 128);
                            store16(Cw, offs, v[j]);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            // fp32 gradients: the same way, 32 columns of 16 rows at a time, which fill the
            // same staging buffers. Rows and columns past the edge get offsets out of range.
            auto store_f32 = [&](float *out, auto add_c) __attribute__((always_inline)) {
                constexpr bool ADD = decltype(add_c)::value;
                // 64 rows of at most 2^25 bytes: offsets below 2^31.
                const __amdgpu_buffer_rsrc_t Cw[2] = {make_rsrc(out + corner, 0x80000000u),
                                                      make_rsrc(out + corner + (size_t)64 * N, 0x80000000u)};
                const uint32_t at0 = (uint32_t)rr * (uint32_t)N * 4u + (uint32_t)rc * 16u;
                constexpr int NF = FM * FN / 2;
                constexpr int AHEAD = 4;   // groups whose old values are on their way
                u32x4 was[AHEAD][2];
#pragma unroll
                for (int gi = 0; gi <= NF; ++gi) {
                    const int fm = gi / (FN / 2), fp = gi % (FN / 2);
                    // Rows 8 j + rr, columns 4 rc .. 4 rc + 3 of group n.
                    auto place = [&](int n, int j) __attribute__((always_inline)) {
                        const int m = n / (FN / 2), p = n % (FN / 2);
                        const bool ok = m * BD + 8 * j + rr < rows_left && p * 32 + 4 * rc < cols_left;
                        return ok ? at0 + (uint32_t)(2 * (m % 4) + j) * 2u * pitch8 + (uint32_t)(p * 128) : kOobOffset;
                    };
                    auto load_was = [&](int n) __attribute__((always_inline)) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            was[n % AHEAD][j] = __builtin_amdgcn_raw_buffer_load_b128(Cw[n / (FN / 2) / 4], (int)place(n, j), 0, 0);
                    };
                    u32x4 v[2];
                    if (gi > 0) {
                        const char *const sb = stg + ((gi - 1) & 1) * STG_BYTES;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            v[j] = *reinterpret_cast<const u32x4 *>(sb + (8 * j + rr) * 128 + ((rc ^ (rr & 7)) * 16));
                    }
                    if constexpr (ADD) {
#pragma unroll
                        for (int n = 0; gi == 0 && n < AHEAD - 1; ++n) load_was(n);
                    }
                    if (gi < NF) {
                        char *const sb = stg + (gi & 1) * STG_BYTES;
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const f32x4 a = value(2 * fp + f, fm);
                            *reinterpret_cast<f32x4 *>(sb + wr * 128 + (((4 * f + wg) ^ (wr & 7)) * 16)) = a;
                        }
                    }
                    if (gi > 0) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            u32x4 o = v[j];
                            if constexpr (ADD) {
                                f32x4 a = __builtin_bit_cast(f32x4, v[j]) + __builtin_bit_cast(f32x4, was[(gi - 1) % AHEAD][j]);
                                o = __builtin_bit_cast(u32x4, a);
                            }
                            __builtin_amdgcn_raw_buffer_store_b128(o, Cw[(gi - 1) / (FN / 2) / 4], (int)place(gi - 1, j), 0, 0);
                        }
                    }
                    if (ADD && gi + AHEAD - 1 < NF) load_was(gi + AHEAD - 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            auto store_tile = [&](auto a_c) __attribute__((always_inline)) {
                if (full)
                    store_all(std::false_type{}, a_c);
                else
                    store_all(std::true_type{}, a_c);
            };
            if constexpr (GRAD) {
                if constexpr (SUMS) {
                    if (with_sums) {
                        // SUMS_A: lane l has the sum of row l % 16 of block f (four times); else
                        // lanes 0, 16, 32, 48 have four columns of block f each.
                        const int width = SUMS_A ? ga->M : N;
                        const int first = SUMS_A ? cur_t.m0 + wm_s * WTM + wr : cur_t.n0 + wn_s * WTN + 4 * wg;
                        const bool add = (ga->flags & GF_ADD) != 0;
#pragma unroll
                        for (int f = 0; f < FM; ++f)
#pragma unroll
                            for (int i = 0; i < (SUMS_A ? 1 : 4); ++i) {
                                const int at = first + f * BD + i;
                                if ((SUMS_A ? wg : wr) != 0 || at >= width) continue;
                                const size_t o = (size_t)cur_t.e * width + at;
                                if constexpr ((ACT & GRAD_F32) != 0) {
                                    float *const p = (float *)ga->sums + o;
                                    *p = add ? *p + sums[f][i] : sums[f][i];
                                } else {
                                    ((uint16_t *)ga->sums)[o] = (uint16_t)pack2<ODT>(sums[f][i], 0.f);
                                }
                            }
                    }
                }
                if constexpr ((ACT & GRAD_F32) != 0) {
                    if (ga->flags & GF_ADD)
                        store_f32((float *)ga->C, std::true_type{});
                    else
                        store_f32((float *)ga->C, std::false_type{});
                } else
                    store_tile(std::integral_constant<int, ACT_NONE>{});
            } else if constexpr (EPI == EPI_SLOPE) {
                store_tile(std::integral_constant<int, ACT_NONE>{});
            } else {
                store_tile(std::integral_constant<int, ACT>{});
            }
        }

        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        if (!nxt_live) break;
        cur_t = nxt_t;
        set_bases(lds_cur - ld_wave);
        read_first();
    }
    wait_vmcnt<0>();   // no direct-to-LDS write may outlive the workgroup's LDS
}

// Grid: one workgroup per CU, or fewer for fewer tiles. Rows mode needs two K
// slices (K > 64 words).
template <int OP, int ODT, int EPI, int ACT, bool TB, bool TA>
hipError_t launch_persist(Group g, hipStream_t stream) {
    const long long tiles_n = ceil_div(g.N, 256);
    const long long row_tiles = TA ? (long long)g.E * ceil_div(g.M, 256) : row_tile_bound(g.T, g.E, 256);
    const long long tiles = row_tiles * tiles_n;
    if (tiles <= 0) return hipSuccess;
    // Tile indices r * G + slot run up to tiles + G - 1: keep them in int.
    if (tiles > 0x7fffffffLL - 0x10000 || (!TA && g.K <= 64)) return hipErrorInvalidValue;
    g.row_bound = (int)row_tiles;
    int cus = 0;
    const hipError_t e = current_cus(&cus);
    if (e != hipSuccess) return e;
    return launch(grouped_persist_kernel<OP, ODT, EPI, ACT, TB, TA>, dim3((unsigned)(tiles < cus ? tiles : cus)), dim3(256),
                  stream, g);
}

}  // namespace gbx
