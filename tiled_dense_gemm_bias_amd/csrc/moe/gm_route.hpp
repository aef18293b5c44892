// Routing to experts: each token's k best of E experts, their weights, and the sorting of the
// (token, expert) slots by expert.
//
// Selection. A row belongs to G lanes (16; 32 from 257 experts on, 64 from 513), lane l holding experts
// l, l + G, ... Each expert's value is a 64-bit float whose low 10 bits are replaced by
// the expert's number, so that one maximum finds the best value and its expert, ties going to the
// lowest number. Without a bias and without sums over groups the value is the logit itself (the
// scores' order, exact in every type); otherwise it is score + bias in 64 bits, cut to 42: values
// that differ by less count as ties. (In 32 bits about one in 10^5 rows of 256 experts chose
// another expert than the formulas do.) A lane sorts its own values once, then k rounds take the
// largest of the G first ones and move up the winner's list. Keys of 32 bits, with the rows done again in 64 whose
// neighbours 32 cannot tell apart, take half the instructions, but the few waves that do both end no sooner.
//
// Groups: the keys go through LDS, where lane g scans group g for its best one or two.
//
// The weights are computed from the chosen logits in 32 bits, renormalised sigmoid weights as
// ratios that do not underflow together: s_i e^-min(m, 0), m the largest chosen logit.
//
// What bounds it: vector instructions, and the latency of small kernels. 16384 rows of 256 fp32 logits with a
// bias, k = 8, are 17 MB (3.3 us at 5.1 TB/s) and take 15 us: 1400 vector instructions a wave of four rows are 70 % of its
// time (a quarter each for the exponentials and the k rounds). 999 rows of grouped experts take 10 us, 8 rows of 32 experts with
// their sorting, all in one workgroup, 3.8 us. As many values in a lane as its registers take (16), as the rounds are a wave's
// and not a value's: 8192 rows of 384 experts take 10.5 us in 32 lanes each and 13.8 in 64 (with a bias 15 and 19).
#pragma once

#include "gm_common.hpp"

namespace gbm {

constexpr int kMaxExperts = 1024, kMaxTop = 32, kMaxGroups = 16;
constexpr int kRouteWaves = 16, kRouteThreads = kRouteWaves * 64;
enum { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1 };

struct Route {
    const void *x;         // [T][E]
    const float *bias;     // [E] or null
    int32_t *indices;      // [T][k]
    float *weights;        // [T][k]
    int32_t *counts;       // [blocks][pitch]: this block's slots of each expert (null: no sort_kernel with several
                           // blocks follows)
    int T, E, k;
    int groups, top_groups, group_best, group_size;
    int score, renorm, dtype;
    float scale;
    int tokens;            // per block
};

// Slots to be sorted by expert: see sort_block.
struct Sort {
    const int32_t *indices;   // [T k]
    const int32_t *counts;    // [blocks][pitch]
    int32_t *offsets;         // [E + 1]
    int32_t *rows;            // [T k]
    int32_t *slots;           // [T k] or null
    int n, E;                 // slots, experts
    int per_block, blocks;    // slots a block
};
__host__ __device__ constexpr int count_pitch(int E) { return (E + 3) & ~3; }   // a block's counts, in whole 16 bytes

constexpr unsigned long long kExpertBits = 1023;

// The value with the expert's number in its low bits: of two equal values the lower number's key is
// the larger. v is finite.
__device__ __forceinline__ double key_of(double v, int e) {
    v += 0.0;   // -0 to +0
    const unsigned long long b = __double_as_longlong(v), low = (unsigned long long)((long long)b < 0 ? e : 1023 - e);
    return __longlong_as_double((long long)((b & ~kExpertBits) | low));
}
__device__ __forceinline__ int expert_of(double key) {
    const long long b = __double_as_longlong(key);
    const int low = (int)(b & (long long)kExpertBits);
    return b < 0 ? low : 1023 - low;
}
__device__ __forceinline__ double without_expert(double key) {
    return __longlong_as_double(__double_as_longlong(key) & ~(long long)kExpertBits);
}

// f over a row's G lanes; every lane gets the result.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const long long b = __double_as_longlong(v);
    const unsigned lo = (unsigned)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xf, 0xf, true);
    const unsigned hi = (unsigned)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xf, 0xf, true);
    return __longlong_as_double((long long)(((unsigned long long)hi << 32) | lo));
}
// The values of this lane and of the one 16 (32) lanes on or back, as a pair.
template <int D>
__device__ __forceinline__ void across(uint32_t v, uint32_t &x, uint32_t &y) {
    const auto s = D == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false) : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    x = s[0];
    y = s[1];
}
template <int D, class F>
__device__ __forceinline__ float join(float v, F f) {
    uint32_t x, y;
    across<D>(__float_as_uint(v), x, y);
    return f(__uint_as_float(x), __uint_as_float(y));
}
template <int D, class F>
__device__ __forceinline__ double join(double v, F f) {
    const long long b = __double_as_longlong(v);
    uint32_t xl, yl, xh, yh;
    across<D>((uint32_t)b, xl, yl);
    across<D>((uint32_t)(b >> 32), xh, yh);
    return f(__longlong_as_double((long long)(((unsigned long long)xh << 32) | xl)), __longlong_as_double((long long)(((unsigned long long)yh << 32) | yl)));
}
template <int G, class T, class F>
__device__ __forceinline__ T all_reduce(T v, F f) {
    v = f(v, dpp<0x128>(v));   // row_ror 8, 4, 2, 1
    v = f(v, dpp<0x124>(v));
    v = f(v, dpp<0x122>(v));
    v = f(v, dpp<0x121>(v));
    if constexpr (G >= 32) v = join<16>(v, f);
    if constexpr (G == 64) v = join<32>(v, f);
    return v;
}
struct Max {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
    __device__ double operator()(double a, double b) const { return __builtin_fmax(a, b); }
};
struct Sum {
    template <class T>
    __device__ T operator()(T a, T b) const { return a + b; }
};
// Whether any of a row's lanes says so. `first`: the row's first lane.
template <int G>
__device__ __forceinline__ bool any_of(bool b, int first) {
    const unsigned long long m = __ballot(b);
    return G == 64 ? m != 0 : ((m >> first) & ((1ull << (G & 63)) - 1)) != 0;
}

// Largest first (Batcher's odd-even merge sort).
template <int P>
__device__ __forceinline__ void sort_keys(double (&v)[P]) {
#pragma unroll
    for (int p = 1; p < P; p *= 2)
#pragma unroll
        for (int q = p; q > 0; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < P; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < P && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const double a = v[i + j], b = v[i + j + q];
                        v[i + j] = __builtin_fmax(a, b);
                        v[i + j + q] = __builtin_fmin(a, b);
                    }
}

// ------------------------------------------------------------------ sorting --

// This block's slots of each expert, for sort_kernel.
__global__ void __launch_bounds__(kRouteThreads)
count_kernel(const int32_t *__restrict__ indices, int32_t *__restrict__ counts, int n, int E, int per_block) {
    __shared__ int count_smem[kMaxExperts];
    const int tid = threadIdx.x;
    for (int e = tid; e < count_pitch(E); e += kRouteThreads) count_smem[e] = 0;
    __syncthreads();
    const long long begin = (long long)blockIdx.x * per_block, end = min((long long)n, begin + per_block);
    for (long long i = begin + tid; i < end; i += kRouteThreads) {
        const int e = indices[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&count_smem[e], 1);
    }
    __syncthreads();
    for (int e = tid; e < count_pitch(E); e += kRouteThreads) counts[(size_t)blockIdx.x * count_pitch(E) + e] = count_smem[e];
}

// Block b sorts its own slots into the rows that its experts' earlier blocks leave: every block adds
// up all blocks' counts (before it: where it starts within an expert; all: the offsets), then its waves
// take equal ranges of its slots in order. Slots of one expert in a wave's 64 find each other by ballots on
// the bits of the expert's number, so that a row's place depends on its slot alone, and on no
// atomic's order. place: LDS, for up to EP experts.
// 131072 slots of 256 experts in 256 blocks take 6.2 us, 8000 in 63 blocks 4.7: a few dependent accesses (half as many
// blocks, with half the counts to read, take as long; experts loaded ahead of the counts 7.3 us).
template <int EP>
__device__ __forceinline__ void sort_block(const Sort &a, int b, int (*place)[EP]) {
    __shared__ int before_smem[EP], total_smem[EP], wave_sum[kRouteWaves];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, E = a.E;
    // ---- counts of all blocks ----
    for (int e = tid; e < EP; e += kRouteThreads) before_smem[e] = total_smem[e] = 0;
    for (int i = tid; i < kRouteWaves * EP; i += kRouteThreads) (&place[0][0])[i] = 0;
    __syncthreads();
    if (a.blocks > 1) {
        // Four experts a thread; the threads past the last four take other blocks of the first ones.
        typedef int i32x4 __attribute__((ext_vector_type(4)));
        const int quads = count_pitch(E) / 4, ways = kRouteThreads / quads;
        const int q = tid % quads, way = tid / quads;
        if (way < ways) {
            i32x4 before = {0, 0, 0, 0}, total = {0, 0, 0, 0};
            const i32x4 *const counts = reinterpret_cast<const i32x4 *>(a.counts) + q;
#pragma unroll 16
            for (int i = way; i < a.blocks; i += ways) {
                const i32x4 c = counts[(size_t)i * quads];
                total += c;
                before += i < b ? c : i32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * q + i < E) {
                    atomicAdd(&before_smem[4 * q + i], before[i]);
                    atomicAdd(&total_smem[4 * q + i], total[i]);
                }
        }
    }
    const long long begin = (long long)b * a.per_block, end = min((long long)a.n, begin + a.per_block);
    // A wave's range: whole rounds of 64.
    const long long each = ((end - begin + kRouteThreads - 1) / kRouteThreads) * 64;
    const long long wbegin = min(begin + wid * each, end), wend = min(wbegin + each, end);
    for (long long i = wbegin + lane; i < wend; i += 64) {
        const int e = a.indices[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&place[wid][e], 1);
    }
    __syncthreads();
    // ---- offsets: a scan over the experts (one a thread), and each wave's first row ----
    static_assert(EP <= kRouteThreads, "one expert a thread");
    int own = 0;
    if (tid < E) {
        if (a.blocks > 1) {
            own = total_smem[tid];
        } else {
#pragma unroll
            for (int w = 0; w < kRouteWaves; ++w) own += place[w][tid];
        }
    }
    int upto = own;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63) wave_sum[wid] = upto;
    __syncthreads();
    int offset = upto - own, all = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
        if (w < wid) offset += wave_sum[w];
        all += wave_sum[w];
    }
    if (tid < E) {
        if (b == 0) a.offsets[tid] = offset;
        int at = offset + before_smem[tid];
#pragma unroll
        for (int w = 0; w < kRouteWaves; ++w) {
            const int c = place[w][tid];
            place[w][tid] = at;
            at += c;
        }
    }
    if (b == 0 && tid == 0) a.offsets[E] = all;
    __syncthreads();
    // ---- each slot's row ----
    const int bits = 32 - __clz(max(E - 1, 1));
    for (long long i0 = wbegin; i0 < wend; i0 += 64) {
        const long long i = i0 + lane;
        int e = -1;
        if (i < wend) e = a.indices[i];
        const bool there = (unsigned)e < (unsigned)E;
        unsigned long long same = __ballot(there);
        for (int bit = 0; bit < bits; ++bit) {
            const unsigned long long set = __ballot((e >> bit) & 1);
            same &= (e >> bit) & 1 ? set : ~set;
        }
        int row = -1;
        if (there) {
            const int at = place[wid][e];
            row = at + __popcll(same & ((1ull << lane) - 1));
            if ((same >> lane) == 1) place[wid][e] = at + __popcll(same);   // its last slot
        }
        wave_sync();
        if (i < wend) {
            a.rows[i] = row;
            if (a.slots && there) a.slots[row] = (int)i;
        }
    }
    // Rows of no slot.
    if (a.slots)
        for (long long i = all + (long long)b * kRouteThreads + tid; i < a.n; i += (long long)a.blocks * kRouteThreads) a.slots[i] = -1;
}

template <int EP>
__global__ void __launch_bounds__(kRouteThreads)
sort_kernel(Sort a) {
    __shared__ int place[kRouteWaves][EP];
    sort_block<EP>(a, blockIdx.x, place);
}

// ------------------------------------------------------------------ routing --

__device__ __forceinline__ float logit(const void *x, int dtype, size_t at) {
    if (dtype == DTYPE_F32) return ((const float *)x)[at];
    const uint32_t h = ((const uint16_t *)x)[at];
    return dtype == DT_BF16 ? to_f32<DT_BF16>(h) : to_f32<DT_F16>(h);
}
// A row's values, `none` past the last. G P experts need no bounds, and a lane's loads then differ by constants only.
template <int G, int P, class T>
__device__ __forceinline__ void load_row(const T *x, int l, int E, T none, T (&v)[P]) {
    const T *const mine = x + l;
    if (E == G * P) {
#pragma unroll
        for (int p = 0; p < P; ++p) v[p] = mine[p * G];
        return;
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        v[p] = none;
        if (p * G + l < E) v[p] = mine[p * G];
    }
}
template <int G, int P>
__device__ __forceinline__ void load_logits(const void *x, int dtype, size_t row, int l, int E, float (&v)[P]) {
    if (dtype == DTYPE_F32) {
        load_row<G, P>((const float *)x + row, l, E, -__builtin_inff(), v);
        return;
    }
    uint16_t h[P];
    load_row<G, P>((const uint16_t *)x + row, l, E, (uint16_t)(dtype == DT_BF16 ? 0xff80 : 0xfc00), h);
#pragma unroll
    for (int p = 0; p < P; ++p) v[p] = dtype == DT_BF16 ? to_f32<DT_BF16>(h[p]) : to_f32<DT_F16>(h[p]);
}

// e^d for d <= 0: the hardware's 2^t with t = d log2 e, what t's rounding lost put back. Within 2^-22; 0 below 2^-126.
__device__ __forceinline__ float exp_neg(float d) {
    const float c = fmaxf(d, -200.0f);   // (-inf: no NaN)
    const float t = c * 1.4426950408889634f;
    const float r = fmaf(c, 1.9259629911e-8f, fmaf(c, 1.4426950408889634f, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, r * 0.6931471805599453f, e);
}

// t_i of the chosen logits (t_i / sum t is the renormalised weight) and, for sigmoid scores,
// s_i e^-min(m, 0) with m the largest: no common underflow.
__device__ __forceinline__ float chosen_score(int score, float x, float m) {
    if (score == SCORE_SOFTMAX) return exp_neg(x - m);
    const float t = exp_neg(-fabsf(x));
    return (x >= 0 ? 1.0f : m >= 0 ? t : exp_neg(x - m)) / (1.0f + t);
}

// p r + c with c in scalar registers (left to itself the compiler copies each c to vector registers for an instruction that
// overwrites it: two more instructions a step).
__device__ __forceinline__ double fma_to(double p, double r, double c) {
    double d;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(p), "v"(r), "s"(c));
    return d;
}

// ln 2 as the 64-bit number nearest to it and the one nearest to what that leaves.
constexpr double kLn2 = 0.6931471805599453, kLn2Rest = 2.3190468138462996e-17;

// e^d for d <= 0 in 64 bits, within 2^-46 (the keys keep 42): d = n ln 2 + r, |r| <= ln 2 / 2 (d - n kLn2 rounds once,
// to 2^-54), and e^r by its series up to r^11 (the next term is 2^-47).
__device__ __forceinline__ double exp_neg(double d) {
    const double c = __builtin_fmax(d, -800.0);
    const double n = __builtin_rint(c * 1.4426950408889634);
    const double r = fma(n, -kLn2Rest, fma(n, -kLn2, c));
    double p = fma(1.0 / 39916800.0, r, 1.0 / 3628800.0);
    p = fma_to(p, r, 1.0 / 362880.0);
    p = fma_to(p, r, 1.0 / 40320.0);
    p = fma_to(p, r, 1.0 / 5040.0);
    p = fma_to(p, r, 1.0 / 720.0);
    p = fma_to(p, r, 1.0 / 120.0);
    p = fma_to(p, r, 1.0 / 24.0);
    p = fma_to(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}
// 1 / d for 1 <= d <= 2^10, within 2^-50: the hardware's 2^-14 or better, by Newton's step, which squares the error, to 2^-28
// and 2^-56; the third leaves its own roundings only, whatever the first is worth.
__device__ __forceinline__ double reciprocal(double d) {
    double q = __builtin_amdgcn_rcp(d);
    q = fma(fma(-d, q, 1.0), q, q);
    q = fma(fma(-d, q, 1.0), q, q);
    return fma(fma(-d, q, 1.0), q, q);
}

// Takes the largest of the row's first keys, `none` if there is none, and moves up that lane's list, of which the first
// D are needed.
template <int G, int D, int P>
__device__ __forceinline__ double take_best(double (&key)[P], double none) {
    const double top = all_reduce<G>(key[0], Max{});
    const bool here = key[0] == top;   // (where there is none left all lists are empty)
    constexpr int N = D < P ? D : P;
#pragma unroll
    for (int p = 0; p + 1 < N; ++p) key[p] = here ? key[p + 1] : key[p];
    key[N - 1] = here ? none : key[N - 1];
    return top;
}

// s.indices: the one block has all tokens and sorts their slots too.
template <int G, int P, bool GROUPED>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(Route a, Sort s) {
    constexpr int RPW = 64 / G;                        // rows a wave
    constexpr int NC = G == 16 ? 2 : 1, EP = G * P;
    const int threads = blockDim.x, RPB = threads / G;  // rows a block and pass
    constexpr bool FUSE = EP <= 256;
    // The rows' keys, where groups are limited; after the rows the sort's places.
    constexpr int KEYS = GROUPED ? kRouteWaves * RPW * EP * 8 : 16, PLACES = FUSE ? kRouteWaves * EP * 4 : 16;
    __shared__ __attribute__((aligned(16))) char smem[KEYS > PLACES ? KEYS : PLACES];
    __shared__ int count_smem[EP];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, sub = lane / G;
    int l = lane & (G - 1);
    const int first = lane - l;
    const double none = -__builtin_inf();
    const long long t0 = (long long)linear_block() * a.tokens;
    const int mine = (int)min((long long)a.tokens, a.T - t0);

    if (a.counts) {
        for (int e = tid; e < a.E; e += threads) count_smem[e] = 0;
        __syncthreads();
    }
    for (int row0 = __builtin_amdgcn_readfirstlane(wid) * RPW; row0 < mine; row0 += RPB) {   // the wave's rows
        const int rr = row0 + sub;
        const bool live = rr < mine;
        const size_t row = (size_t)(t0 + (live ? rr : 0)) * a.E;
        asm volatile("" : "+v"(l));   // else the biases and the experts' groups stay in registers from pass to pass, and these run out
        float x[P];
        load_logits<G, P>(a.x, a.dtype, row, l, a.E, x);
        const bool softmax = a.score == SCORE_SOFTMAX;
        const bool scored = a.bias != nullptr || (GROUPED && a.group_best > 1);
        float b[P];
        if (a.bias) {
            load_row<G, P>(a.bias, l, a.E, 0.0f, b);
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p) b[p] = 0.0f;
        }
        float m = -__builtin_inff();
        bool bad = false;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            m = fmaxf(m, x[p]);
            bad |= x[p] != x[p] || b[p] != b[p];
            b[p] = fminf(b[p], 3.4e38f);   // finite, beside a masked logit's -inf
        }
        if (softmax) {
            m = all_reduce<G>(m, Max{});
            bad |= m == __builtin_inff();
        }
        bad = any_of<G>(bad, first);

        // ---- keys ----
        __builtin_amdgcn_sched_barrier(0);
        float z = 0.0f;      // softmax: the sum of e^(x - m)
        double key[P];
        if (scored) {
            double sum = 0.0;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const double t = exp_neg(softmax ? (double)x[p] - (double)m : -__builtin_fabs((double)x[p]));
                key[p] = softmax ? t : (x[p] >= 0 ? 1.0 : t) * reciprocal(1.0 + t);
                if (x[p] == -__builtin_inff()) key[p] = none;
                sum += __builtin_fmax(key[p], 0.0);
                __builtin_amdgcn_sched_barrier(0);   // one after the other: side by side they take too many registers
            }
            double by = 1.0;
            if (softmax) {
                sum = all_reduce<G>(sum, Sum{});
                z = (float)sum;
                by = sum > 0.0 ? reciprocal(sum) : 1.0;
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                key[p] = fma(key[p], by, (double)b[p]);   // -inf is `none`, a bias's too
            }
        } else {
            if (softmax && !a.renorm) {
#pragma unroll
                for (int p = 0; p < P; ++p) z += x[p] == -__builtin_inff() ? 0.0f : exp_neg(x[p] - m);
                z = all_reduce<G>(z, Sum{});
            }
#pragma unroll
            for (int p = 0; p < P; ++p) key[p] = __builtin_fmin((double)x[p], 1e300);   // (sigmoid: +inf)
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
            key[p] = bad || key[p] == none ? none : key_of(key[p], p * G + l);

        // ---- groups ----
        if constexpr (GROUPED) {
            double *const mykeys = reinterpret_cast<double *>(smem) + (wid * RPW + sub) * EP;
#pragma unroll
            for (int p = 0; p < P; ++p) mykeys[p * G + l] = key[p];
            wave_sync();
            double best = none, next = none;
            if (l < a.groups)
#pragma unroll 4
                for (int i = 0, c = l % a.group_size; i < a.group_size; ++i) {
                    const double v = mykeys[l * a.group_size + c];
                    next = __builtin_fmax(next, __builtin_fmin(best, v));
                    best = __builtin_fmax(best, v);
                    if (++c == a.group_size) c = 0;   // each group from another start: other banks
                }
            double total = best == none ? none : without_expert(best);
            if (a.group_best > 1 && next != none) total += without_expert(next);
            int better = 0;
            for (int i = 0; i < a.groups; ++i) {
                const double o = __shfl(total, first + i);
                better += o > total || (o == total && i < l);
            }
            const unsigned long long kept = __ballot(l < a.groups && better < a.top_groups) >> first;
            const unsigned magic = ((1u << 20) + a.group_size - 1) / a.group_size;   // e / group_size = e magic >> 20
#pragma unroll
            for (int p = 0; p < P; ++p)   // (read again, not held meanwhile)
                key[p] = (kept >> (((unsigned)(p * G + l) * magic) >> 20)) & 1 ? mykeys[p * G + l] : none;
            wave_sync();
        }

        // ---- the k best ----
        __builtin_amdgcn_sched_barrier(0);
        sort_keys(key);
        __builtin_amdgcn_sched_barrier(0);
        int chosen[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) chosen[c] = -1;
        const auto choose = [&](auto depth_c) __attribute__((always_inline)) {
            for (int j = 0; j < a.k; ++j) {
                const double top = take_best<G, decltype(depth_c)::value>(key, none);
                const int e = top == none ? -1 : expert_of(top);
                if (l == j) chosen[0] = e;
                if constexpr (NC == 2)
                    if (l + 16 == j) chosen[1] = e;
            }
        };
        if (P > 8 && a.k <= 8)   // shorter lists to move up
            choose(std::integral_constant<int, 8>{});
        else
            choose(std::integral_constant<int, P>{});

        // ---- their weights ----
        float xs[NC], w[NC];
        float mc = -__builtin_inff();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const bool there = live && l + c * G < a.k && chosen[c] >= 0;
            xs[c] = there ? logit(a.x, a.dtype, row + chosen[c]) : -__builtin_inff();
            mc = fmaxf(mc, xs[c]);
        }
        if (a.renorm) mc = all_reduce<G>(mc, Max{});
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const bool there = live && l + c * G < a.k && chosen[c] >= 0;
            w[c] = there ? chosen_score(a.score, xs[c], a.renorm ? mc : a.score == SCORE_SOFTMAX ? m : 0.0f) : 0.0f;
            sum += w[c];
        }
        if (a.renorm)
            sum = all_reduce<G>(sum, Sum{});
        else
            sum = a.score == SCORE_SOFTMAX ? z : 1.0f;
        const float by = sum > 0.0f ? a.scale / sum : 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int j = l + c * G;
            if (live && j < a.k) {
                const size_t at = (size_t)(t0 + rr) * a.k + j;
                a.indices[at] = chosen[c];
                a.weights[at] = bad ? __builtin_nanf("") : w[c] * by;
                if (a.counts && chosen[c] >= 0) atomicAdd(&count_smem[chosen[c]], 1);
            }
        }
    }
    if (a.counts) {
        __syncthreads();
        int32_t *const counts = a.counts + (size_t)blockIdx.x * count_pitch(a.E);
        for (int e = tid; e < count_pitch(a.E); e += threads) counts[e] = e < a.E ? count_smem[e] : 0;
    }
    if constexpr (FUSE) {
        if (s.indices) {
            __syncthreads();   // the chosen experts are in memory
            sort_block<EP>(s, 0, reinterpret_cast<int(*)[EP]>(smem));
        }
    }
}

// ----------------------------------------------------------------- gradient --

struct RouteGrad {
    const void *x;
    const int32_t *indices;
    const float *dw;
    void *dx;
    int T, E, k;
    int score, renorm, dtype;
    float scale;
};

constexpr int kGradWaves = 4;

// With g = scale dw and D the sum of (weight / scale) g over the chosen:
//   softmax, renormalised:  dx_i = q_i (g_i - D) for the chosen, q the softmax over them; else 0
//   softmax:                dx_e = p_e (g_e [chosen] - D) for every expert
//   sigmoid, renormalised:  dx_i = q_i (1 - s_i) (g_i - D)
//   sigmoid:                dx_i = g_i s_i (1 - s_i)
// Only softmax that is not renormalised reads all logits of a row; so do rows without any slot, for a NaN among them.
// A row's chosen terms go through LDS to the lanes that hold the experts; reading and writing the logits
// and their gradient once is what bounds it (16384 x 256 in fp32 8.3 us, 4.1 TB/s; renormalised 7.5).
template <int G, int P>
__global__ void __launch_bounds__(kGradWaves * 64)
route_grad_kernel(RouteGrad a) {
    constexpr int RPW = 64 / G, NC = G == 16 ? 2 : 1;
    __shared__ float smem[kGradWaves * RPW][G * P];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int l = lane & (G - 1), first = lane - l;
    const long long t = ((long long)linear_block() * kGradWaves + wid) * RPW + lane / G;
    const bool live = t < a.T;
    const size_t row = (size_t)(live ? t : 0) * a.E;
    float *const terms = smem[wid * RPW + lane / G];
#pragma unroll
    for (int p = 0; p < P; ++p) terms[p * G + l] = 0.0f;
    int e[NC];
    float g[NC], xs[NC], mc = -__builtin_inff();
    bool some = false;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int j = l + c * G;
        e[c] = -1;
        if (live && j < a.k) e[c] = a.indices[(size_t)t * a.k + j];
        if ((unsigned)e[c] >= (unsigned)a.E) e[c] = -1;
        const bool there = e[c] >= 0;
        g[c] = there ? a.scale * a.dw[(size_t)t * a.k + j] : 0.0f;
        xs[c] = there ? logit(a.x, a.dtype, row + e[c]) : -__builtin_inff();
        mc = fmaxf(mc, xs[c]);
        some |= there;
    }
    some = any_of<G>(some, first);
    const bool dense = a.score == SCORE_SOFTMAX && !a.renorm;
    float x[P], m = -__builtin_inff(), z = 0.0f;
    if (dense || !some) load_logits<G, P>(a.x, a.dtype, row, l, a.E, x);
    // A row without any slot: NaN where moe_route's weights are, else zeros.
    float none = 0.0f;
    if (!some) {
        bool bad = false;
#pragma unroll
        for (int p = 0; p < P; ++p) bad |= x[p] != x[p] || (a.score == SCORE_SOFTMAX && x[p] == __builtin_inff());
        none = any_of<G>(bad, first) ? __builtin_nanf("") : 0.0f;
    }
    if (dense) {
#pragma unroll
        for (int p = 0; p < P; ++p) m = fmaxf(m, x[p]);
        m = all_reduce<G>(m, Max{});
#pragma unroll
        for (int p = 0; p < P; ++p) {
            x[p] = x[p] == -__builtin_inff() ? 0.0f : exp_neg(x[p] - m);
            z += x[p];
        }
        z = all_reduce<G>(z, Sum{});
    } else {
        m = all_reduce<G>(mc, Max{});
    }
    float q[NC], sum = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        q[c] = e[c] >= 0 ? chosen_score(a.score, xs[c], a.renorm || dense ? m : 0.0f) : 0.0f;
        sum += q[c];
    }
    sum = all_reduce<G>(sum, Sum{});
    const float by = dense ? 1.0f / z : a.renorm ? 1.0f / sum : 1.0f;
    float d = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        q[c] *= by;
        if (e[c] >= 0) d = fmaf(q[c], g[c], d);
    }
    d = dense || a.renorm ? all_reduce<G>(d, Sum{}) : 0.0f;
    wave_sync();
    bool again = false;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (e[c] < 0) continue;
        float v = g[c];
        if (!dense) v = q[c] * (v - d);
        if (a.score == SCORE_SIGMOID) v *= chosen_score(SCORE_SIGMOID, -xs[c], 0.0f);   // 1 - s
        q[c] = v;
        again |= atomicAdd(&terms[e[c]], v) != 0.0f;   // a repeated expert's terms add up
    }
    wave_sync();
    if (any_of<G>(again, first)) {
        // Of an expert that is there more than once: in the order of its slots, not in the atomics'.
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (e[c] >= 0) terms[e[c]] = 0.0f;
        wave_sync();
#pragma unroll
        for (int c = 0; c < NC; ++c)
            for (int j = 0; j < G && c * G + j < a.k; ++j) {
                if (l == j && e[c] >= 0) terms[e[c]] += q[c];
                wave_sync();
            }
    }
    if (!live) return;
    float v[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        v[p] = terms[p * G + l];
        if (dense) v[p] = x[p] * by * (v[p] - d);
        v[p] = some ? v[p] : none;
    }
    const auto store = [&](auto dtype_c) __attribute__((always_inline)) {
        constexpr int DT = decltype(dtype_c)::value;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const size_t at = row + p * G + l;
            if (p * G + l >= a.E) continue;
            if constexpr (DT == DTYPE_F32)
                ((float *)a.dx)[at] = v[p];
            else
                ((uint16_t *)a.dx)[at] = (uint16_t)pack2<DT>(v[p], 0.0f);
        }
    };
    if (a.dtype == DTYPE_F32)
        store(std::integral_constant<int, DTYPE_F32>{});
    else if (a.dtype == DT_BF16)
        store(std::integral_constant<int, DT_BF16>{});
    else
        store(std::integral_constant<int, DT_F16>{});
}

}  // namespace gbm
