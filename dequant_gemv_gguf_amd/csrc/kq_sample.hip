// kq_sample.hip -- a token for each row of logits (include/kqstep.h).
//
// Everything that the filters leave is a leading part of the tokens in the order
// of (logit descending, index ascending), so a filter is a place in that order.
//
// Bound: for few rows the chain of two launches (one row of 32000 tokens, top_k 40,
// top_p and min_p: 13 us); for many the arithmetic of the first (256 rows of 151937,
// settings of each row: 76 us, of which it takes 52; 3.0 TB/s there, 6.8 where all rows
// are greedy).  Two launches:
//  * chunk_kernel, a work-group a chunk of 8192 tokens of a row: the chunk's first
//    token of the order, a histogram over bins of an eighth of an octave of weight
//    (counts and weights of 512 bins below the chunk's largest), and a list of its
//    first tokens.  The bins lie at fixed places of l / t, so chunks need not know of
//    each other.  A bin's count and the sum of its weights, integers, share one
//    64-bit LDS atomic: the sums do not depend on the order.  The count that a token
//    finds there is its place in its bin, so that the chunk can also leave its tokens
//    ordered by bins.
//  * row_kernel, a work-group a row: the chunks' histograms added up give the bin in
//    which each filter ends.  Where few tokens are left down to that bin (hundreds,
//    and all in the chunks' lists), every one of them is compared with every other
//    and that is all (one row of 32000 13 us; by digits, as below, 20).  Elsewhere
//    the bin's tokens are gathered from the ordered chunks into registers (256 rows
//    76 us; by a scan of the row 84), the place among them is found digit by digit of the
//    logits' keys, the chunks' kept weights say which chunk holds the token, and its
//    logits are gone over once more.  Bins of more than 6144 tokens (thousands of equal
//    logits, a very high temperature) are not kept: the row is read for every digit, of
//    11 bits there (one row of 151937 equal logits 400 us; of 8 bits 730).
// Weights are 2^(l log2(e) / t) with 36 bits of mantissa, relative to the octave of
// the row's largest: a chunk's 8192 of them and their count are one 64-bit word, and a
// probability, rounded to 2^-24, has 2^12 steps of them to a step of its own.
#include "kq_step.h"

#include <cmath>
#include <type_traits>

namespace kq {
namespace step {

constexpr int CHUNK_THREADS = 512, CHUNK = 8192;
constexpr int ROW_THREADS = 1024, ROW_WAVES = ROW_THREADS / 64;
constexpr int MAX_V = 1 << 20, MAX_CHUNKS = MAX_V / CHUNK;
constexpr int BINS = 512, OCTAVE = 8;             // bins, and those of an octave
constexpr int COUNT_SHIFT = 50;                   // a bin: count, and below it the sum of weights
constexpr int LIST = 6144;                        // tokens that row_kernel keeps in registers
constexpr int NEAR = 256;                         // tokens of a chunk's list
constexpr int SPARSE = 1024;                      // tokens of a chunk that can matter, where those are put together first
constexpr int FEW = 256;                          // tokens that are compared with each other
constexpr int SLICE = 16384;                      // chunks of a launch, or one row: 390 MB of workspace
static_assert((u64)CHUNK << 37 <= 1ull << COUNT_SHIFT, "a chunk's weights fit a bin's sum");

struct Sample {
    const float *logits, *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *tokens;
    float *probs;
    u64 *tops;              // [row][chunk] first token
    u32 *near_n;            // [row][chunk] tokens of its list
    u64 *near;              // [row][chunk][NEAR]
    u64 *hist;              // [row][chunk][BINS]
    uint16_t *upto;         // [row][chunk][BINS] tokens down to and with a bin
    uint16_t *order;        // [row][chunk][CHUNK] and their places, bin after bin
    int64_t ld;
    int V, chunks, row0;    // (the launch's first row; the workspace's rows are counted from it)
};

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

// The key of a logit, in the logits' order: 0 for what is never taken.  (+ 0: the
// zeros are equal.)  A token: its key, and the lower index first.
__device__ __forceinline__ u32 key_of(float l) {
    const u32 b = __builtin_bit_cast(u32, l + 0.f);
    return l > -__builtin_inff() ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float logit_of(u32 key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ u64 token_of(u32 key, int i) { return (u64)key << 32 | (u32)~i; }

// Where a logit's weight lies: the bin (counted upwards), its octave, and the
// mantissa, 2^35 .. 2^36.  (A bin is the nearest whole number to what is 1/2 less than
// the eighths of an octave.)  What is left of the logit is one product and sum, so that
// it is off by 2^-54 of a bin however far from 0 the logits lie (as the difference of the
// rounded eighths and the bin it was off by 2^-54 of the eighths: a weight by 2^-27 at
// l / t of 2^27).
struct Scale {
    double eighths, quarters;   // of an octave, per logit: 8 log2(e) / t, and half of it
    const double *steps;        // 2^(35 + (i + 1/2) / 8), i < 8, in LDS
    // (an infinite logit's bin is given by what it is compared with)
    __device__ __forceinline__ double bin(float l) const { return rint(fma((double)l, eighths, -0.5)); }
    // that of a first token: an infinite one lies above all others
    __device__ __forceinline__ double top_bin(float l) const { return l < __builtin_inff() ? bin(l) : __builtin_inf(); }
    // 2^52 more, in whose low bits it is rounded to an integer.  `of_octave`: the bin's
    // place in its octave
    __device__ __forceinline__ double mantissa_d(float l, int of_octave) const {
        // half of what is left, from the bin's middle at 1/2: 1/4 .. 3/4, and a rounding of
        // the bin more.  (Past 2^35 bins, or where it is no number, only equal logits are in
        // one, and any value does: 0 .. 1, which costs no instruction and lets sums be
        // 2^(1/16) as large.)
        const double y = fmin(fmax(fma((double)l, quarters, fma(bin(l), -0.5, 0.25)), 0.0), 1.0);
        // 2^((2 y - 1) / 8) by the polynomial through six Chebyshev nodes: off by 2^-41
        double p = 0x1.5d8dfde822453p-20;
        p = fma(p, y, 0x1.1fe3316ea9487p-15);
        p = fma(p, y, 0x1.a0ff35b3145fdp-11);
        p = fma(p, y, 0x1.c326766be389ep-7);
        p = fma(p, y, 0x1.456fd368e4058p-3);
        p = fma(p, y, 0x1.d5818dcc704b1p-1);
        return fma(p, steps[of_octave], 0x1p52);
    }
    // `plus` 2^32 more
    __device__ __forceinline__ u64 mantissa(float l, int of_octave, u32 plus = 0) const {
        const u64 b = __builtin_bit_cast(u64, mantissa_d(l, of_octave));
        return (u64)((u32)(b >> 32) - 0x43300000u + plus) << 32 | (u32)b;
    }
};
__device__ __forceinline__ Scale scale_of(float t, const double *steps) {
    const double quarters = t < __builtin_inff() ? 4.0 * 1.4426950408889634 / (double)t : 0.0;
    return Scale{2.0 * quarters, quarters, steps};
}
__device__ const double STEPS[OCTAVE] = {0x1.0b5586cf9890fp+35, 0x1.2387a6e756238p+35, 0x1.3dea64c123422p+35, 0x1.5ab07dd485429p+35,
                                         0x1.7a11473eb0187p+35, 0x1.9c49182a3f090p+35, 0x1.c199bdd85529cp+35, 0x1.ea4afa2a490dap+35};
// from mod OCTAVE, of the first token's bin (an infinite one: the octave's last)
__device__ __forceinline__ int phase_of(double from) {
    return from < __builtin_inf() ? (int)(from - OCTAVE * floor(from / OCTAVE)) : OCTAVE - 1;
}

// Logits i .. i + 3 of a row, -infinity past its end.
__device__ __forceinline__ f4 four(const float *l, int i, int V) {
    f4 x;
    if (i + 4 <= V) {
        x = *(const f4u *)(l + i);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = i + j < V ? l[min(i + j, V - 1)] : -__builtin_inff();
    }
    return x;
}

// A load that stays where it is written: others are put off until past the first
// return, and then wait behind what they could have been on their way with.
template <class N> __device__ __forceinline__ N at_once(const N *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
}

// A row's settings, all on their way at once (what is not given is read where u is).
struct Settings {
    float t, top_p, min_p, u;
    int top_k;
};
__device__ __forceinline__ Settings settings_of(const Sample &a, int row) {
    const float t = (a.temperature ? a.temperature : a.u)[row], p = (a.top_p ? a.top_p : a.u)[row], m = (a.min_p ? a.min_p : a.u)[row];
    const int k = (a.top_k ? a.top_k : (const int32_t *)a.u)[row];
    return Settings{a.temperature ? t : 1.f, a.top_p ? p : 1.f, a.min_p ? m : 0.f, a.u[row], a.top_k ? k : 0};
}

// Across lanes, by DPP: the value of another lane, or `none` where there is none.
template <int CTRL, int ROWS> __device__ __forceinline__ u32 dpp_or(u32 none, u32 x) {
    return (u32)__builtin_amdgcn_update_dpp((int)none, (int)x, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS> __device__ __forceinline__ u64 dpp_or(u64 none, u64 x) {
    return (u64)dpp_or<CTRL, ROWS>((u32)(none >> 32), (u32)(x >> 32)) << 32 | dpp_or<CTRL, ROWS>((u32)none, (u32)x);
}
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_or(double none, double x) {
    return __builtin_bit_cast(double, dpp_or<CTRL, ROWS>(__builtin_bit_cast(u64, none), __builtin_bit_cast(u64, x)));
}
template <int CTRL, int ROWS> __device__ __forceinline__ float dpp_or(float none, float x) {
    return __builtin_bit_cast(float, dpp_or<CTRL, ROWS>(__builtin_bit_cast(u32, none), __builtin_bit_cast(u32, x)));
}
// Inclusive sums over a wave; op over a wave, in every lane.
template <class N> __device__ __forceinline__ N wave_scan(N x) {
    x += dpp_or<0x111, 0xF>(N(0), x);
    x += dpp_or<0x112, 0xF>(N(0), x);
    x += dpp_or<0x114, 0xF>(N(0), x);
    x += dpp_or<0x118, 0xF>(N(0), x);
    x += dpp_or<0x142, 0xA>(N(0), x);
    x += dpp_or<0x143, 0xC>(N(0), x);
    return x;
}
__device__ __forceinline__ u32 last_lane(u32 x) { return (u32)__builtin_amdgcn_readlane((int)x, 63); }
__device__ __forceinline__ u64 last_lane(u64 x) { return (u64)last_lane((u32)(x >> 32)) << 32 | last_lane((u32)x); }
__device__ __forceinline__ float last_lane(float x) { return __builtin_bit_cast(float, last_lane(__builtin_bit_cast(u32, x))); }
__device__ __forceinline__ double last_lane(double x) { return __builtin_bit_cast(double, last_lane(__builtin_bit_cast(u64, x))); }
template <class N, class Op> __device__ __forceinline__ N wave_all(N x, Op op) {
    x = op(x, dpp_or<0x111, 0xF>(x, x));
    x = op(x, dpp_or<0x112, 0xF>(x, x));
    x = op(x, dpp_or<0x114, 0xF>(x, x));
    x = op(x, dpp_or<0x118, 0xF>(x, x));
    x = op(x, dpp_or<0x142, 0xA>(x, x));
    x = op(x, dpp_or<0x143, 0xC>(x, x));
    return last_lane(x);
}
__device__ __forceinline__ u64 wave_max(u64 x) {
    return wave_all(x, [](u64 p, u64 q) { return p > q ? p : q; });
}
// x summed over the lanes of a quad.
__device__ __forceinline__ u64 quad_sum(u64 x) {
    x += dpp_or<0xB1, 0xF>(0ull, x);
    return x + dpp_or<0x4E, 0xF>(0ull, x);
}

// Room for n things of each lane in a list whose length is *count: where the lane's
// begin.
__device__ __forceinline__ int room(int *count, int n) {
    const int upto = (int)wave_scan((u32)n), all = (int)last_lane((u32)upto);
    int at = 0;
    if (all && (threadIdx.x & 63) == 63) at = atomicAdd(count, all);
    return __builtin_amdgcn_readlane(at, 63) + upto - n;
}

// Whether top_k limits the row (the same in both kernels).
__device__ __forceinline__ bool limited(int top_k, int V) { return top_k > 0 && top_k < V; }

// Bound: its arithmetic, some 30 instructions a token whose weight is asked for, 15 of
// them in 64 bits (256 rows of 151937 that all sum weights: 58 us, without the weights
// 44, greedy 23).  top_k up to the threads of a work-group, and min_p alone, first take
// out the tokens that cannot matter and count the others, put together in LDS (256 rows
// 76 us, 84 where top_k counts them all; top_k 50 alone 39 and 60).
__global__ __launch_bounds__(CHUNK_THREADS) void chunk_kernel(const Sample a) {
    constexpr int PER = CHUNK / CHUNK_THREADS, WAVES = CHUNK_THREADS / 64;
    constexpr float LEAST = -3.402823466e38f;     // the least logit that counts
    // two histograms, of the even and the odd lanes: half the lanes of a wave meet in a bin
    __shared__ __align__(16) u64 hist[BINS][2];
    __shared__ uint16_t some[SPARSE];             // places in the chunk
    __shared__ float tops[WAVES], floors[WAVES];
    __shared__ u32 counts[WAVES];
    __shared__ double steps[OCTAVE];
    __shared__ __align__(16) uint16_t order[CHUNK];
    __shared__ u32 starts[BINS];                  // where a bin's even lanes' tokens begin in `order`, and from bit 16 its odd lanes'
    __shared__ int n_some, n_near, n_all, first_most;
    const int row = a.row0 + blockIdx.y, chunk = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const float *l = a.logits + row * a.ld;
    const Settings set = settings_of(a, row);
    const double step = STEPS[tid & (OCTAVE - 1)];
    const float t = set.t, top_p = set.top_p, min_p = set.min_p;
    const int top_k = set.top_k;
    const int base = chunk * CHUNK;
    auto place = [&](int i) { return 4 * tid + 4 * CHUNK_THREADS * (i / 4) + i % 4; };
    float v[PER];
#pragma unroll
    for (int p = 0; p < PER; p += 4) {
        const f4 x = four(l, base + place(p), a.V);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[p + j] = x[j];
    }
    for (int i = tid; i < 2 * BINS; i += CHUNK_THREADS) (&hist[0][0])[i] = 0;
    if (tid == 0) {
        n_some = n_near = n_all = 0;
        first_most = INT32_MAX;
    }
    if (tid < OCTAVE) steps[tid] = step;
    const float none = -__builtin_inff();
    float mine = none;                            // (a NaN is never the larger one)
#pragma unroll
    for (int i = 0; i < PER; ++i) mine = fmaxf(mine, v[i]);
    // Logits below `floor` cannot be among the first top_k: so many groups of lanes
    // have a greater one.
    const bool by_k = limited(top_k, a.V);
    float floor_ = mine;
    if (by_k && top_k <= CHUNK_THREADS / 2) floor_ = fmaxf(floor_, dpp_or<0xB1, 0xF>(floor_, floor_));
    if (by_k && top_k <= CHUNK_THREADS / 4) floor_ = fmaxf(floor_, dpp_or<0x4E, 0xF>(floor_, floor_));
    if (by_k && top_k <= CHUNK_THREADS / 8) floor_ = fmaxf(floor_, dpp_or<0x141, 0xF>(floor_, floor_));
    floor_ = wave_all(floor_, [](float p, float q) { return fminf(p, q); });
    float most = wave_all(mine, [](float p, float q) { return fmaxf(p, q); });
    if (lane == 0) {
        tops[tid >> 6] = most;
        floors[tid >> 6] = floor_;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        most = fmaxf(most, tops[w]);
        floor_ = fminf(floor_, floors[w]);
    }
    const int64_t at = (int64_t)blockIdx.y * a.chunks + chunk;
    if (!(most > none)) {
        if (tid == 0) a.tops[at] = 0;
        return;
    }
    if (mine == most) {
        int i = PER - 1;
#pragma unroll
        for (int j = PER - 2; j >= 0; --j) i = v[j] == most ? j : i;
        atomicMin(&first_most, base + place(i));
    }
    if (!(t > 0.f)) {
        __syncthreads();
        if (tid == 0) a.tops[at] = token_of(key_of(most), first_most);
        return;
    }
    const Scale s = scale_of(t, steps);
    const double from = s.top_bin(most);
    const int phase = phase_of(from);
    bool sparse = by_k && top_k <= CHUNK_THREADS;
    if (!by_k && !(top_p < 1.f) && min_p > 0.f) {
        // with min_p alone: nor can logits of less than that part of the largest weight (and a little less)
        const float x = most + t * fminf(logf(min_p), 0.f);
        floor_ = x - (fabsf(most) + fabsf(x)) * 0x1p-18f - 1e-30f;
        sparse = true;
    }
    floor_ = sparse ? fmaxf(floor_, LEAST) : LEAST;
    auto bin_of = [&](float x) {
        const double d = fmin(from - s.bin(x), BINS - 1.0);
        return x == most ? 0 : (int)d;
    };
    // returns the bin, and below bit 16 the tokens that its half had before
    auto count = [&](float x) {
        const int b = bin_of(x);
        // (with top_k no weights are asked for, and never those of the last bin, 64 octaves below)
        constexpr u32 ONE = 1u << (COUNT_SHIFT - 32);
        const u64 w = by_k ? (u64)ONE << 32 : s.mantissa(x, (phase - b) & (OCTAVE - 1), ONE);
        return (u32)b << 16 | (u32)(atomicAdd((unsigned long long *)&hist[b][lane & 1], w) >> COUNT_SHIFT);
    };
    if (sparse) {
        u32 mask = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) mask |= (u32)(v[i] >= floor_) << i;
        int to = room(&n_some, __popc(mask));
        for (; mask; mask &= mask - 1, ++to)
            if (to < SPARSE) some[to] = (uint16_t)place(__builtin_ctz(mask));
        __syncthreads();
        sparse = n_some <= SPARSE;
    }
    float x[SPARSE / CHUNK_THREADS];              // (read again: a lane's logits cannot be picked by number)
    int some_at[SPARSE / CHUNK_THREADS];
    u32 where[PER];                               // what `count` returned; ~0: not counted
    if (sparse) {
#pragma unroll
        for (int i = 0; i < SPARSE / CHUNK_THREADS; ++i) {
            const bool in = tid + i * CHUNK_THREADS < n_some;
            some_at[i] = in ? some[tid + i * CHUNK_THREADS] : 0;
            x[i] = in ? l[base + some_at[i]] : none;
        }
#pragma unroll
        for (int i = 0; i < SPARSE / CHUNK_THREADS; ++i) {
            where[i] = ~0u;
            if (x[i] > none) where[i] = count(x[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            where[i] = ~0u;
            if (v[i] >= floor_) where[i] = count(v[i]);
        }
    }
    // (a row without filters needs neither its chunks' order nor their lists)
    const bool ordered = by_k || top_p < 1.f || min_p > 0.f;
    __syncthreads();
    const u64 even = hist[tid][0], h = even + hist[tid][1];
    a.hist[at * BINS + tid] = h;
    u32 upto = wave_scan((u32)(h >> COUNT_SHIFT));
    if (lane == 63) counts[tid >> 6] = upto;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES - 1; ++w) upto += w < tid >> 6 ? counts[w] : 0;
    if (ordered) {
        const u32 start = upto - (u32)(h >> COUNT_SHIFT);
        starts[tid] = start | (start + (u32)(even >> COUNT_SHIFT)) << 16;
        a.upto[at * BINS + tid] = (uint16_t)upto;
        if (tid == BINS - 1) n_all = (int)upto;
    }
    // the list: whole bins from the top, as many as fit
    const int depth = __syncthreads_count(upto <= NEAR);
    if (ordered) {
        // a place for each token from its bin and the count that it found there
        auto put = [&](u32 where, int i) {
            const u32 from = starts[where >> 16];
            const int to = (int)(lane & 1 ? from >> 16 : from & 0xFFFF) + (int)(where & 0xFFFF);
            order[to] = (uint16_t)i;
            return to;
        };
        if (sparse) {
#pragma unroll
            for (int i = 0; i < SPARSE / CHUNK_THREADS; ++i)
                if (where[i] != ~0u) {
                    const int to = put(where[i], some_at[i]);
                    if ((int)(where[i] >> 16) < depth) a.near[at * NEAR + to] = token_of(key_of(x[i]), base + some_at[i]);
                }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (where[i] != ~0u) put(where[i], place(i));
        }
        if (tid == depth - 1) n_near = (int)upto;
    }
    __syncthreads();
    if (ordered) {
        for (int i = tid; 8 * i < n_all; i += CHUNK_THREADS) ((uint4 *)(a.order + at * CHUNK))[i] = ((const uint4 *)order)[i];
        if (!sparse && tid < n_near) {
            const int i = base + order[tid];
            a.near[at * NEAR + tid] = token_of(key_of(l[i]), i);
        }
    }
    if (tid == 0) {
        a.tops[at] = token_of(key_of(most), first_most);
        a.near_n[at] = (u32)n_near;
    }
}
static_assert(NEAR <= CHUNK_THREADS, "a thread a token of the list");
static_assert(FEW <= NEAR, "where a row has so few down to a bin, its chunks' lists go down to it");
static_assert(CHUNK_THREADS == BINS, "a thread a bin");

// Bits by which the sum of n weights of 36 bits of mantissa can be finer than these.
constexpr int FINEST = 27;
__host__ __device__ constexpr int finer_for(int n) {
    int bits = 0;
    while (n > 1 << bits) ++bits;
    return FINEST - bits;
}
constexpr int FEW_FINER = finer_for(FEW);

// Bits of a digit where the tokens are in registers, and where the row is read for each.
constexpr int DIGIT = 8, WIDE_DIGIT = 11;
static_assert(1 << WIDE_DIGIT == 2 * ROW_THREADS, "two digits a thread");

// What row_kernel shares between its threads.
struct RowSpace {
    struct { u64 token, weight; } few[FEW];
    u32 begin[MAX_CHUNKS], skip[MAX_CHUNKS];        // of a chunk's gathered tokens among all; and to their places in its order
    u64 weight[BINS];               // of the row's bins
    double upto[BINS];              // summed weights up to and with a bin, in units of the top octave's mantissas
    u32 count[BINS], counts[BINS];  // tokens of a bin, and up to and with it
    u64 digit_weight[1 << WIDE_DIGIT];
    u32 digit_count[1 << WIDE_DIGIT];
    u64 chunk_list[MAX_CHUNKS];     // kept weight of a chunk's gathered tokens
    double chunk_sum[MAX_CHUNKS];
    u64 waves[ROW_WAVES];
    double waves_d[ROW_WAVES];
    u64 found[3];                   // a digit, what lies above it, its tokens
    double picked[2];
    u64 most, sum;
    double steps[OCTAVE];
    int off[MAX_CHUNKS];            // bins that a chunk's are below the row's (BINS: all of them; -1: it has no token)
    int n, low, high;
};

// One row of logits as every thread of row_kernel sees it.
struct Row {
    const float *l;
    Scale s;
    u64 best;               // the first token of the order
    double from;            // its bin
    int phase;              // from mod OCTAVE
    double least;           // min_p: the least weight kept
    // bin b (downwards from the top's) is this many octaves below the top's octave
    __device__ __forceinline__ int octaves(int b) const { return (b + OCTAVE - 1 - phase) >> 3; }
    __device__ __forceinline__ int bin(float x) const {
        if (x == logit_of((u32)(best >> 32))) return 0;
        return (int)fmin(from - s.bin(x), (double)BINS);
    }
    // in units of the top octave's mantissas; 0 past the bin `last`, at most BINS - 2
    __device__ __forceinline__ double weight(float x, int last) const {
        const int b = bin(x);
        const double w = ldexp(s.mantissa_d(x, (phase - b) & (OCTAVE - 1)) - 0x1p52, -octaves(b));
        return b <= last ? w : 0.0;
    }
    __device__ __forceinline__ u64 mantissa(float x, int b) const { return s.mantissa(x, (phase - b) & (OCTAVE - 1)); }
    // whether min_p keeps it (by its whole weight: `integer` loses bits of small ones)
    __device__ __forceinline__ bool keeps(u64 token) const {
        return !(least > 0.0) || token == best || weight(logit_of((u32)(token >> 32)), BINS - 2) >= least;
    }
    // as an integer, in units of the mantissas `base` octaves below, 2^finer to one; at
    // least 1 (a u of 0 takes the first token that is kept, however little it weighs)
    __device__ __forceinline__ u64 integer(u64 token, int finer, int base) const {
        const float x = logit_of((u32)(token >> 32));
        const int b = bin(x), down = min(octaves(b) - base, 63);
        return b < BINS - 1 ? max((mantissa(x, b) << finer) >> down, (u64)1) : 0;
    }
};

// The shortest leading part (descending) of the tokens from `from` on that `each` goes
// over, of which the counts, or the weights (WEIGHTS), sum to at least `want` (1 .. the
// whole sum): the part is the tokens from the returned place on (which need not be a
// token).  Digits of what a token is above `from` (to find the bits in which they differ
// instead takes two reductions and 1.5 us), from the first that one up to `top`, the
// most that any is, can have.  The digits' sums are 0 before and after.
template <bool WEIGHTS, bool WIDE, class Each>
__device__ __forceinline__ u64 cut(RowSpace &m, Each &&each, u64 from, u64 top, u64 want) {
    constexpr int BITS = WIDE ? WIDE_DIGIT : DIGIT, INDEX = 20;
    static_assert(MAX_V == 1 << INDEX, "");
    const int tid = threadIdx.x, lane = tid & 63;
    if (WIDE) {
        // (equal logits are common, and would all meet in a digit: the first of the bits
        // in which the keys differ)
        u32 most = 0, least = 0;
        each([&](u64 token, auto &&) {
            if (token < from) return;
            most = max(most, (u32)(token >> 32));
            least = max(least, ~(u32)(token >> 32));
        });
        auto larger = [](u32 p, u32 q) { return max(p, q); };
        most = wave_all(most, larger);
        least = wave_all(least, larger);
        __syncthreads();                    // (waves may still read the last block_sum's there)
        if (lane == 0) m.waves[tid >> 6] = (u64)most << 32 | least;
        __syncthreads();
        for (int w = 0; w < ROW_WAVES; ++w) {
            most = max(most, (u32)(m.waves[w] >> 32));
            least = max(least, (u32)m.waves[w]);
        }
        from = max(from, (u64)~least << 32);
        top = min(top, (u64)most << 32 | 0xFFFFFFFF);
        __syncthreads();
    }
    // (wide, with the index in 20 bits: fewer digits)
    auto over = [&](u64 token) {
        return WIDE ? (u64)((u32)(token >> 32) - (u32)(from >> 32)) << INDEX | (token & (MAX_V - 1)) : token - from;
    };
    const u64 most = top > from ? over(top) : 0;
    int above = most ? 64 - __builtin_clzll(most) : 0;                     // bits from here on are `prefix`
    u64 prefix = 0, before = 0;
    while (above) {
        const int shift = max(above - BITS, 0);
        const u32 digits = (1u << (above - shift)) - 1;
        each([&](u64 token, auto &&weight) {
            const u64 v = over(token);
            if (token < from || (above < 64 && v >> above != prefix)) return;
            const u32 d = (u32)(v >> shift) & digits;
            atomicAdd(&m.digit_count[d], 1u);
            if (WEIGHTS) atomicAdd((unsigned long long *)&m.digit_weight[d], weight());
        });
        __syncthreads();
        // EACH digits a lane, descending, by one wave or by all
        constexpr int EACH = WIDE ? 2 : 4;
        u32 n[EACH];
        u64 d[EACH], s = 0, upto = 0;
        if (WIDE || tid < 64) {
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const int digit = (1 << BITS) - 1 - (EACH * tid + i);
                n[i] = m.digit_count[digit];
                d[i] = WEIGHTS ? m.digit_weight[digit] : n[i];
                m.digit_count[digit] = 0;
                if (WEIGHTS) m.digit_weight[digit] = 0;
                s += d[i];
            }
            upto = wave_scan(s);
        }
        bool here;
        if (WIDE) {
            if (lane == 63) m.waves[tid >> 6] = upto;
            __syncthreads();
            for (int w = 0; w < tid >> 6; ++w) upto += m.waves[w];
            upto += before;
            here = upto >= want ? upto - s < want : tid == ROW_THREADS - 1;
        } else {
            upto += before;
            const u64 reach = __ballot(upto >= want);
            here = tid < 64 && lane == (reach ? __builtin_ctzll(reach) : 63);
        }
        if (here) {
            u64 b = upto - s;
            int at = 0;
            u32 count = n[0];
#pragma unroll
            for (int i = 0; i < EACH - 1; ++i)
                if (at == i && b + d[i] < want) {
                    b += d[i];
                    at = i + 1;
                    count = n[i + 1];
                }
            m.found[0] = (u64)((1 << BITS) - 1 - (EACH * tid + at));
            m.found[1] = b;
            m.found[2] = count;
        }
        __syncthreads();
        prefix = prefix << (above - shift) | m.found[0];
        before = m.found[1];
        above = shift;
        if (m.found[2] == 1) break;         // one token has these digits: none lies between it and them
    }
    const u64 v = prefix << above;
    if (!WIDE) return from + v;
    return max(from, (u64)((u32)(from >> 32) + (u32)(v >> INDEX)) << 32 | (0xFFFFFFFFu - (MAX_V - 1)) | (v & (MAX_V - 1)));
}

__device__ __forceinline__ u64 block_sum(RowSpace &m, u64 x) {
    const int tid = threadIdx.x, lane = tid & 63;
    x = wave_scan(x);
    __syncthreads();
    if (lane == 63) m.waves[tid >> 6] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < ROW_WAVES; ++w) x += m.waves[w];
    return x;
}

__global__ __launch_bounds__(ROW_THREADS) void row_kernel(const Sample a) {
    __shared__ RowSpace m;
    const int row = a.row0 + blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Settings set = settings_of(a, row);
    const double step = STEPS[tid & (OCTAVE - 1)];
    const float t = set.t, top_p = set.top_p, min_p = set.min_p;
    const int top_k = set.top_k;
    const int64_t chunk0 = (int64_t)blockIdx.x * a.chunks;
    // What a wave needs first is asked for at once: the histograms of two chunks, the
    // list of one.  (Not all of it was written: a chunk without a token has neither, a
    // list is as long as near_n says.)
    u64 bins[2][BINS / 64], listed_[NEAR / 64];
    auto ask_bins = [&](int k, int c) {
        if (c >= a.chunks) return;
        const u64 *h = a.hist + (chunk0 + c) * BINS;
#pragma unroll
        for (int i = 0; i < BINS / 64; ++i) bins[k][i] = at_once(h + lane + 64 * i);
    };
    auto ask_list = [&](int c) {
        if (c >= a.chunks) return;
        const u64 *from = a.near + (chunk0 + c) * NEAR;
#pragma unroll
        for (int i = 0; i < NEAR / 64; ++i) listed_[i] = at_once(from + lane + 64 * i);
    };
    // a lane's chunks: c = lane, lane + 64
    u64 first_of[MAX_CHUNKS / 64], best = 0;
    u32 near_n[MAX_CHUNKS / 64];
#pragma unroll
    for (int i = 0; i < MAX_CHUNKS / 64; ++i) {
        const int64_t c = chunk0 + min(lane + 64 * i, a.chunks - 1);
        first_of[i] = at_once(a.tops + c);
        near_n[i] = at_once(a.near_n + c);
    }
    if (t > 0.f) {
        ask_bins(0, wave);
        ask_bins(1, wave + ROW_WAVES);
        ask_list(wave);
    }
#pragma unroll
    for (int i = 0; i < MAX_CHUNKS / 64; ++i) {
        if (lane + 64 * i >= a.chunks) first_of[i] = near_n[i] = 0;
        best = first_of[i] > best ? first_of[i] : best;
    }
    best = wave_max(best);
    if (!(best >> 32) || !(t > 0.f)) {
        if (tid == 0) {
            a.tokens[row] = best >> 32 ? (int)~(u32)best : -1;
            if (a.probs) a.probs[row] = best >> 32 ? 1.f : 0.f;
        }
        return;
    }
    Row r;
    r.l = a.logits + row * a.ld;
    r.s = scale_of(t, m.steps);
    r.best = best;
    const float most = logit_of((u32)(best >> 32));
    r.from = r.s.top_bin(most);
    r.phase = phase_of(r.from);

    // the row's histogram
    for (int b = tid; b < BINS; b += ROW_THREADS) {
        m.weight[b] = 0;
        m.count[b] = 0;
    }
    if (tid < 1 << DIGIT) {
        m.digit_weight[tid] = 0;
        m.digit_count[tid] = 0;
    }
    if (tid == 0) {
        m.n = 0;
        m.low = BINS;
        m.high = -1;
    }
    if (wave == 0) {
#pragma unroll
        for (int i = 0; i < MAX_CHUNKS / 64; ++i) {
            const int c = lane + 64 * i;
            const u32 key = (u32)(first_of[i] >> 32);
            const float x = logit_of(key);
            const double d = x == most ? 0.0 : r.from - r.s.top_bin(x);
            m.off[c] = !key ? -1 : (int)fmin(d, (double)BINS);
            m.chunk_list[c] = 0;
        }
        if (lane == 0) m.most = m.sum = 0;
    }
    if (tid < OCTAVE) m.steps[tid] = step;
    __syncthreads();
    r.least = min_p > 0.f ? (double)min_p * (double)r.mantissa(most, 0) : 0.0;
    for (int c0 = wave; c0 < a.chunks; c0 += 2 * ROW_WAVES) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = c0 + k * ROW_WAVES, off = c < a.chunks ? m.off[c] : -1;
            if (off < 0) continue;
#pragma unroll
            for (int i = 0; i < BINS / 64; ++i) {
                const u64 x = bins[k][i];
                if (!x) continue;
                const int b = min(lane + 64 * i + off, BINS - 1);
                atomicAdd(&m.count[b], (u32)(x >> COUNT_SHIFT));
                const u64 w = x & ((1ull << COUNT_SHIFT) - 1);
                if (w && b < BINS - 1) atomicAdd((unsigned long long *)&m.weight[b], w);
            }
        }
        ask_bins(0, c0 + 2 * ROW_WAVES);
        ask_bins(1, c0 + 3 * ROW_WAVES);
    }
    __syncthreads();
    {
        // sums over the bins from the top
        u32 n = 0;
        double w = 0.0;
        if (tid < BINS) {
            n = wave_scan(m.count[tid]);
            w = wave_scan(ldexp((double)m.weight[tid], -r.octaves(tid)));
            if (lane == 63) {
                m.waves[wave] = n;
                m.waves_d[wave] = w;
            }
        }
        __syncthreads();
        if (tid < BINS) {
            for (int v = 0; v < wave; ++v) {
                n += (u32)m.waves[v];
                w += m.waves_d[v];
            }
            m.counts[tid] = n;
            m.upto[tid] = w;
        }
        __syncthreads();
    }
    const int total = (int)m.counts[BINS - 1];
    const bool by_k = limited(top_k, a.V), by_p = top_p < 1.f;
    const int keep_k = min(top_k, total);         // (fewer than top_k tokens may be above -infinity)
    const double all = m.upto[BINS - 1], want_p = (double)(top_p > 0.f ? top_p : 0.f) * all;
    // the bins in which top_k, top_p and min_p end
    if (tid < BINS) {
        const u32 n0 = tid ? m.counts[tid - 1] : 0, n1 = m.counts[tid];
        const double w0 = tid ? m.upto[tid - 1] : 0.0, w1 = m.upto[tid];
        if (by_k) {
            if ((int)n0 < keep_k && (int)n1 >= keep_k) m.low = tid;
        } else if (by_p && (tid == 0 || w0 < want_p) && (w1 >= want_p || tid == BINS - 1)) {
            atomicMin(&m.low, tid);
        }
    }
    __syncthreads();
    int low = m.low, high = low;                  // the tokens of bins high .. low decide
    if (!by_k && r.least > 0.0) {
        // The bin of the least weight; those above it are kept whole.  A token's bin is that
        // of its rounded eighths of an octave, off by up to 2^-53 of them, and its weight by
        // 2^-35: where the least weight is so near to a border, both bins' tokens decide.
        // (Equal logits past all bins may weigh a little more than their bin: none of them
        // but the first is left above 1, nor is one where an infinite min_p makes a bin a NaN.)
        const double at = OCTAVE * (log2(r.least) - 35.0), near = fmin(0x1p-31 + (fabs(r.from) + BINS) * 0x1p-52, 0x1p-8);
        auto bin_of = [&](double at) {
            const double b = r.phase - floor(at);
            return !(b >= 0.0) ? 0 : b < BINS ? (int)b : BINS - 1;
        };
        const int first = min_p > 1.f ? 0 : bin_of(at + near), last = min_p > 1.f ? 0 : bin_of(at - near);
        if (first <= low) {
            high = first;
            low = min(low, last);
        }
    }
    const bool one = !by_k && low < BINS;         // (mostly one bin)
    // (the last bin's tokens weigh nothing: what ends there leaves all the others)
    if (low == BINS - 1) low = BINS - 2;
    high = by_k ? 0 : min(high, low);
    if (low < BINS && m.counts[low] <= FEW) {
        // Few tokens, all of them in the chunks' lists: each with those before it (4 threads
        // a token, a quarter of the others each).
        for (int c = wave; c < a.chunks; c += ROW_WAVES) {
            if (c != wave) ask_list(c);
            if (m.off[c] < 0 || m.off[c] > low) continue;
            const int n = __builtin_amdgcn_readlane((int)(c < 64 ? near_n[0] : near_n[1]), c & 63);
            u32 mask = 0;
#pragma unroll
            for (int i = 0; i < NEAR / 64; ++i) mask |= (u32)(lane + 64 * i < n && r.bin(logit_of((u32)(listed_[i] >> 32))) <= low) << i;
            int to = room(&m.n, __popc(mask));
#pragma unroll
            for (int i = 0; i < NEAR / 64; ++i)
                if (mask >> i & 1) {
                    if (to < FEW) m.few[to].token = listed_[i];
                    ++to;
                }
        }
        __syncthreads();
        // (a wave has 16 tokens; those without any only wait)
        const int n = min(m.n, FEW), i = tid >> 2, part = tid & 3;
        const bool any = 16 * wave < n;
        u64 token = 0, weight = 0, upto = 0, place = 0;
        if (any) {
            token = m.few[min(i, n - 1)].token;
            weight = r.integer(token, FEW_FINER, 0);
            if (i < n && part == 0) m.few[i].weight = weight;
        }
        __syncthreads();
        bool kept = false;
        if (any) {
#pragma unroll 4
            for (int j = part; j < n; j += 4) {
                const bool before = m.few[j].token >= token;
                place += before;
                upto += before ? m.few[j].weight : 0;
            }
            place = quad_sum(place);
            upto = quad_sum(upto);
            kept = i < n && (!by_k || (int)place <= keep_k);
            const u64 mine = wave_max(kept ? upto : 0);
            if (lane == 0) atomicMax((unsigned long long *)&m.most, mine);
        }
        __syncthreads();
        if (any) {
            if (by_p) {
                const double want = by_k ? (double)(top_p > 0.f ? top_p : 0.f) * (double)m.most : ldexp(want_p, FEW_FINER);
                kept = kept && (place == 1 || (double)(upto - weight) < want);
            }
            kept = kept && r.keeps(token);
            const u64 mine = wave_max(kept ? upto : 0);
            if (lane == 0) atomicMax((unsigned long long *)&m.sum, mine);
            if (i < n && part == 0 && !kept) m.few[i].weight = 0;
        }
        __syncthreads();
        if (!any) return;
        // the kept weights up to each token, by index
        const u64 sum = m.sum;
        const float u = set.u;
        const double at = (u > 0.f ? (double)u : 0.0) * (double)sum;
        const u64 past = at < (double)sum ? min((u64)at, sum - 1) : sum - 1;
        u64 before = 0;
#pragma unroll 4
        for (int j = part; j < n; j += 4) before += (u32)m.few[j].token > (u32)token ? m.few[j].weight : 0;
        before = quad_sum(before);
        if (part == 0 && kept && before <= past && past < before + weight) {
            a.tokens[row] = (int)~(u32)token;
            if (a.probs) a.probs[row] = (float)(r.weight(logit_of((u32)(token >> 32)), BINS - 2) / ldexp((double)sum, -FEW_FINER));
        }
        return;
    }
    // bins high .. low are gathered
    const u32 gathered = low < BINS ? m.counts[low] - (high ? m.counts[high - 1] : 0) : 0;
    const bool scan = low < BINS;
    // what can lie in these bins, and a little more
    float lo = -3.402823466e38f, hi = __builtin_inff();
    if (r.s.eighths > 0.0 && most < __builtin_inff()) {
        const double x = (r.from - low) / r.s.eighths;
        lo = fmaxf(lo, (float)(x - fabs(x) * 0x1p-22) - 1e-37f);
        const double y = (r.from - high + 1) / r.s.eighths;
        hi = (float)(y + fabs(y) * 0x1p-22) + 1e-37f;
    }
    const bool listed = scan && gathered <= LIST;
    // Weights of gathered tokens as integers: with one bin (or two) in units of its octave's
    // mantissas, which hold them whole (the second's with a bit more); else of the top's,
    // and finer by the bits that the sum of so many of at most 2^36 leaves of 63.
    const int base = one ? r.octaves(high) : 0, down = one ? r.octaves(low) - base : 0;
    int finer = finer_for(listed ? LIST : (int)gathered);
    u64 least = 0;                                // top_k and top_p keep the tokens from here on
    // each(f): f(token, weight()) for every gathered token; wide: from the row
    auto places = [&](auto &&each, auto wide) {
        constexpr bool WIDE = decltype(wide)::value;
        // (where the tokens of these bins lie)
        const u64 lowest = (u64)key_of(lo) << 32, top = min(best, (u64)key_of(hi) << 32 | 0xFFFFFFFF);
        if (by_k && (int)m.counts[low] >= top_k) least = cut<false, WIDE>(m, each, lowest, top, (u64)top_k);
        u64 sum = one ? (m.weight[low] << finer >> down) + (high < low ? m.weight[high] << finer : 0) : 0;
        if (by_k && WIDE) {
            // (many tokens may weigh little together: as fine as their sum lets)
            finer = FINEST;
            unsigned __int128 mine = 0;
            each([&](u64 token, auto &&weight) {
                if (token >= least) mine += weight();
            });
            const u64 low48 = block_sum(m, (u64)mine & ((1ull << 48) - 1)), above = block_sum(m, (u64)(mine >> 48)) + (low48 >> 48);
            const int drop = max(48 + 64 - (above ? __builtin_clzll(above) : 64) - 63, 0);
            finer -= drop;
            sum = (u64)(((unsigned __int128)above << 48 | (low48 & ((1ull << 48) - 1))) >> drop);
        } else if (by_k && by_p) {
            u64 mine = 0;
            each([&](u64 token, auto &&weight) { mine += token >= least ? weight() : 0; });
            sum = block_sum(m, mine);
        }
        if (by_p && (by_k || low == m.low)) {
            // of what top_k leaves; in the bin that decides, what the bins above it leave
            const double want = one ? ldexp(want_p - (high ? m.upto[high - 1] : 0.0), base + finer)
                                    : (double)(top_p > 0.f ? top_p : 0.f) * (double)sum;
            least = cut<true, WIDE>(m, each, max(least, lowest), top, want > 1.0 ? (want < (double)sum ? (u64)ceil(want) : sum) : 1);
        }
        __syncthreads();
        // kept weight of the gathered tokens, by chunk (wide: a thread's tokens of a chunk
        // follow each other, and all lanes are at the same one)
        u64 mine = 0;
        int at = 0;
        auto put = [&] {
            if (mine) atomicAdd((unsigned long long *)&m.chunk_list[at], mine);
            mine = 0;
        };
        each([&](u64 token, auto &&weight) {
            if (token < least) return;
            const int c = (int)~(u32)token / CHUNK;
            const u64 w = weight();
            if (!w || !r.keeps(token)) return;
            if (WIDE && c != at) put();
            at = c;
            mine += w;
            if (!WIDE) put();
        });
        put();
        __syncthreads();
    };
    if (listed) {
        // Bins high .. low of each chunk, one behind the other: where each begins, and
        // where the chunk's order has it.
        if (wave == 0) {
            u32 before = 0;
#pragma unroll
            for (int i = 0; i < MAX_CHUNKS / 64; ++i) {
                const int c = lane + 64 * i, off = m.off[c];
                const uint16_t *upto = a.upto + (chunk0 + c) * BINS;
                const bool in = off >= 0 && off <= low;
                const u32 from = in && high > off ? upto[high - off - 1] : 0, n = (in ? upto[low - off] : 0) - from;
                const u32 all = wave_scan(n);
                m.begin[c] = before + all - n;
                m.skip[c] = from - m.begin[c];
                before += last_lane(all);
            }
        }
        __syncthreads();
        // A thread's tokens and their weights, in registers (0: none).  (Of 1024 tokens the
        // lanes of a wave take those 65 apart, which lie in several chunks: their sums
        // below would wait for one address.)
        constexpr int TOKENS = LIST / ROW_THREADS, HALF = TOKENS / 2;
        u64 token[TOKENS], w[TOKENS];
        const int n = (int)gathered;
#pragma unroll
        for (int h = 0; h < TOKENS; h += HALF) {
#pragma unroll
            for (int i = h; i < h + HALF; ++i) token[i] = w[i] = 0;
            if (h * ROW_THREADS >= n) continue;
            int at[HALF];
            float x[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
                const int first = (h + i) * ROW_THREADS, p = min(first + (first + ROW_THREADS <= n ? (tid * 65) & (ROW_THREADS - 1) : tid), n - 1);
                int c = 0;
#pragma unroll
                for (int step = MAX_CHUNKS / 2; step; step >>= 1)
                    if (step < a.chunks && c + step < a.chunks && (int)m.begin[c + step] <= p) c += step;
                at[i] = c * CHUNK + a.order[(chunk0 + c) * CHUNK + p + (int)m.skip[c]];
            }
#pragma unroll
            for (int i = 0; i < HALF; ++i) x[i] = r.l[at[i]];
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
                const int first = (h + i) * ROW_THREADS;
                if (first >= n || (first + ROW_THREADS > n && first + tid >= n)) continue;
                token[h + i] = token_of(key_of(x[i]), at[i]);
                w[h + i] = r.integer(token[h + i], finer, base);
            }
        }
        places([&](auto &&f) {
#pragma unroll
            for (int i = 0; i < LIST / ROW_THREADS; ++i)
                if (i * ROW_THREADS < n && token[i]) f(token[i], [&] { return w[i]; });
        }, std::false_type());
    } else if (scan) {
        for (int i = tid; i < 1 << WIDE_DIGIT; i += ROW_THREADS) {
            m.digit_weight[i] = 0;
            m.digit_count[i] = 0;
        }
        if (one && high < low) {
            // two bins: their first and last logits
            u32 first = key_of(lo), last = key_of(fminf(hi, most));
            for (u32 end = last; first < end;) {
                const u32 at = first + (end - first) / 2;
                if (r.bin(logit_of(at)) <= low) end = at;
                else first = at + 1;
            }
            for (u32 from = first; from < last;) {
                const u32 at = last - (last - from) / 2;
                if (r.bin(logit_of(at)) >= high) from = at;
                else last = at - 1;
            }
            lo = logit_of(first);
            hi = logit_of(last);
        }
        // (the next logits are on their way)
        auto row = [&](auto &&f) {
            f4 now = four(r.l, 4 * tid, a.V);
            for (int i = 4 * tid; i < a.V; i += 4 * ROW_THREADS) {
                const f4 next = four(r.l, i + 4 * ROW_THREADS, a.V);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (now[j] >= lo && now[j] <= hi) f(now[j], token_of(key_of(now[j]), i + j));
                now = next;
            }
        };
        if (one && high == low) {
            // one bin: its mantissas are the weights
            const double bin = r.from - low;
            const int of_octave = (r.phase - low) & (OCTAVE - 1);
            places([&](auto &&f) {
                row([&](float x, u64 token) {
                    if (x == most ? low == 0 : r.s.bin(x) == bin) f(token, [&] { return r.s.mantissa(x, of_octave) << finer; });
                });
            }, std::true_type());
        } else {
            places([&](auto &&f) {
                row([&](float x, u64 token) {
                    // (with top_k a token a rounding past bin `low` is past the last one that it keeps)
                    f(token, [&] { return r.integer(token, finer, base); });
                });
            }, std::true_type());
        }
    }
    // and of the bins above them
    const int whole = !scan ? BINS : one ? high : 0;
    for (int c0 = wave; c0 < a.chunks; c0 += 2 * ROW_WAVES) {
        int off[2];
        u64 h[2][BINS / 64];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = c0 + k * ROW_WAVES;
            off[k] = c < a.chunks ? __builtin_amdgcn_readfirstlane(m.off[c]) : -1;
            if (off[k] < 0) off[k] = BINS;
#pragma unroll
            for (int i = 0; i < BINS / 64; ++i) h[k][i] = off[k] + 64 * i < whole ? a.hist[(chunk0 + c) * BINS + lane + 64 * i] : 0;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = c0 + k * ROW_WAVES;
            if (c >= a.chunks) break;
            double w = 0.0;
#pragma unroll
            for (int i = 0; i < BINS / 64; ++i) {
                if (off[k] + 64 * i >= whole) break;
                const int b = off[k] + 64 * i + lane;
                const double x = ldexp((double)(h[k][i] & ((1ull << COUNT_SHIFT) - 1)), -r.octaves(b));
                w += b < min(whole, BINS - 1) ? x : 0.0;
            }
            w = sum_d<64>(w);
            if (lane == 0) m.chunk_sum[c] = w + ldexp((double)m.chunk_list[c], -base - finer);
        }
    }
    __syncthreads();
    // the chunk
    if (wave == 0) {
        constexpr int EACH = MAX_CHUNKS / 64;
        double s[EACH], mine = 0.0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            s[i] = EACH * lane + i < a.chunks ? m.chunk_sum[EACH * lane + i] : 0.0;
            mine += s[i];
        }
        const double upto = wave_scan(mine), sum = last_lane(upto);
        const float u = set.u;
        const double at = (u > 0.f ? fmin((double)u, 1.0) : 0.0) * sum;
        // the first lane whose sum passes `at`, else the last that has any weight
        const u64 past = __ballot(upto > at && mine > 0.0), some = __ballot(mine > 0.0);
        const int who = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
        if (lane == who) {
            double b = upto - mine;
            int i = 0;
            for (int j = 1; j < EACH; ++j)
                if (s[j] > 0.0 && (s[i] <= 0.0 || b + s[i] <= at)) {
                    b += s[i];
                    i = j;
                }
            m.n = EACH * lane + i;
            m.picked[0] = at - b;
            m.picked[1] = sum;
            m.low = a.V;
            m.high = -1;
        }
    }
    __syncthreads();
    // Its token.  Where its chunk keeps up to half of its tokens down to bin `low`, these
    // alone, by their places' upper bits and then one by one; else all of the chunk's (8
    // rows of 128256 22 us, with all of the chunk's 23.4; with a quarter, half or three
    // quarters as the limit they are even, and 256 of 151937 within 1 %).
    const int64_t chosen = chunk0 + m.n;
    const int below = low - m.off[m.n], kept_n = scan && below >= 0 ? a.upto[chosen * BINS + below] : CHUNK;
    constexpr int EVERY = 4, PIECES = 256, PIECE = CHUNK / PIECES;
    if (kept_n <= EVERY * ROW_THREADS) {
        constexpr int FINER = finer_for(EVERY * ROW_THREADS);
        const int top = r.octaves(m.off[m.n]);    // (of the chunk's own first token)
        int at[EVERY];
        u64 w[EVERY];
#pragma unroll
        for (int j = 0; j < EVERY; ++j) at[j] = a.order[chosen * CHUNK + min(tid + j * ROW_THREADS, kept_n - 1)];
#pragma unroll
        for (int j = 0; j < EVERY; ++j) {
            w[j] = 0;
            if (64 * wave + j * ROW_THREADS >= kept_n) continue;
            const int i = m.n * CHUNK + at[j];
            const u64 token = token_of(key_of(r.l[i]), i);
            if (tid + j * ROW_THREADS < kept_n && token >= least && r.keeps(token)) w[j] = r.integer(token, FINER, top);
            if (w[j]) atomicAdd((unsigned long long *)&m.digit_weight[at[j] / PIECE], w[j]);
        }
        if (tid < PIECE) m.digit_weight[PIECES + tid] = 0;
        __syncthreads();
        if (wave == 0) {
            u64 d[PIECES / 64], s = 0;
#pragma unroll
            for (int i = 0; i < PIECES / 64; ++i) s += d[i] = m.digit_weight[PIECES / 64 * lane + i];
            const u64 upto = wave_scan(s), all = last_lane(upto);
            u64 past = m.picked[0] > 0.0 ? (u64)fmin(ldexp(m.picked[0], FINER + top), 0x1.fffffffffffffp63) : 0;
            past = past < all ? past : all - 1;
            const u64 reach = __ballot(all && upto > past);
            if (lane == (reach ? __builtin_ctzll(reach) : 0)) {
                u64 b = upto - s;
                int i = 0;
                for (; i < PIECES / 64 - 1 && b + d[i] <= past; ++i) b += d[i];
                m.found[0] = all ? (u64)(PIECES / 64 * lane + i) : PIECES;
                m.found[1] = past - b;
            }
        }
        __syncthreads();
        const int piece = (int)m.found[0];
#pragma unroll
        for (int j = 0; j < EVERY; ++j)
            if (w[j] && at[j] / PIECE == piece) m.digit_weight[PIECES + at[j] % PIECE] = w[j];
        __syncthreads();
        if (wave == 0) {
            const u64 mine = lane < PIECE ? m.digit_weight[PIECES + lane] : 0, upto = wave_scan(mine);
            const u64 hit = __ballot(mine && upto > m.found[1]);
            // (weights that differ by a rounding left none: the row's first)
            if (lane == (hit ? __builtin_ctzll(hit) : 0)) {
                const int token = hit ? m.n * CHUNK + piece * PIECE + lane : (int)~(u32)best;
                a.tokens[row] = token;
                if (a.probs) a.probs[row] = (float)(r.weight(r.l[token], BINS - 2) / m.picked[1]);
            }
        }
        return;
    }
    constexpr int EACH = CHUNK / ROW_THREADS;
    const int first = m.n * CHUNK + EACH * tid;
    const double at = m.picked[0], sum = m.picked[1];
    f4 logits[EACH / 4];
#pragma unroll
    for (int j = 0; j < EACH / 4; ++j) logits[j] = four(r.l, first + 4 * j, a.V);
    // (`least` as a logit and an index; no token's key lies below that of the lowest
    // number, or at that of -0)
    u32 last_key = (u32)(least >> 32), last_low = (u32)least;
    if (last_key == 0x7FFFFFFF) {
        last_key = 0x80000000;
        last_low = 0;
    }
    const float last_x = last_key >= 0x00800000 ? logit_of(last_key) : -__builtin_inff();
    const int last_i = last_key >= 0x00800000 ? (int)min(~last_low, 0x7FFFFFFFu) : -1, best_i = (int)~(u32)best;
    // (nothing past bin `low` is kept, also where `least` lies there)
    const int last_bin = min(low, BINS - 2);
    double w[EACH] = {}, mine = 0.0;
    if (m.n * CHUNK + EACH * 64 * wave < a.V) {
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
            // (a weight for every token, also those that are not kept: without branches the
            // eight are computed side by side)
            const float x = logits[j / 4][j % 4];
            w[j] = r.weight(x, last_bin);
            const int kept = ((x > last_x) | ((x == last_x) & (first + j <= last_i))) & ((first + j == best_i) | (w[j] >= r.least));
            w[j] = kept ? w[j] : 0.0;
            mine += w[j];
        }
    }
    double upto = wave_scan(mine);
    if (lane == 63) m.waves_d[wave] = upto;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < ROW_WAVES; ++v) upto += v < wave ? m.waves_d[v] : 0.0;
    double b = upto - mine;
    int token = a.V, last = -1;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        b += w[j];
        if (w[j] > 0.0) {
            last = first + j;
            if (b > at && token == a.V) token = first + j;
        }
    }
    // (the wave's first and last ones: in LDS a thousand lanes would wait for one address)
    const u64 here = __ballot(token < a.V), any = __ballot(last >= 0);
    if (here && lane == __builtin_ctzll(here)) atomicMin(&m.low, token);
    if (any && lane == 63 - __builtin_clzll(any)) atomicMax(&m.high, last);
    __syncthreads();
    token = m.low < a.V ? m.low : m.high;
    if (token < 0) {                              // (weights that differ by a rounding left none: the row's first)
        if (tid == 0) {
            a.tokens[row] = best_i;
            if (a.probs) a.probs[row] = (float)(r.weight(most, 0) / sum);
        }
        return;
    }
    if (token >= first && token < first + EACH) {
        double p = 0.0;
#pragma unroll
        for (int j = 0; j < EACH; ++j) p = first + j == token ? w[j] : p;
        a.tokens[row] = token;
        if (a.probs) a.probs[row] = (float)(p / sum);
    }
}

// The parts of a workspace, for `rows` rows at a time.
struct SampleSpace { size_t near_n, near, hist, upto, order, end; int chunks, rows; };
static SampleSpace sample_space(int M, int64_t V) {
    SampleSpace s;
    s.chunks = (int)((V + CHUNK - 1) / CHUNK);
    s.rows = std::max(1, std::min(M, SLICE / s.chunks));
    const size_t n = (size_t)(M ? s.rows : 0) * s.chunks;
    s.near_n = n * sizeof(u64);
    s.near = (s.near_n + n * sizeof(u32) + 15) & ~(size_t)15;
    s.hist = s.near + n * NEAR * sizeof(u64);
    s.upto = s.hist + n * BINS * sizeof(u64);
    s.order = s.upto + n * BINS * sizeof(uint16_t);
    s.end = s.order + n * CHUNK * sizeof(uint16_t);
    return s;
}

} // namespace step
} // namespace kq

using namespace kq;
using namespace kq::step;

extern "C" {

size_t kqstep_sample_workspace_bytes(int M, int64_t V) {
    if (M < 0 || M > 65536 || V < 1 || V > MAX_V) return 0;
    return sample_space(M, V).end;
}

int kqstep_sample(int M, int64_t V, const float *logits, int64_t ld, const float *temperature, const int32_t *top_k,
                  const float *top_p, const float *min_p, const float *u, int32_t *tokens, float *probs, void *workspace,
                  size_t workspace_bytes, void *stream) {
    if (M < 0 || M > 65536 || V < 1 || V > MAX_V || ld < V || ld > ((int64_t)1 << 40)) return KQ_ERR_SHAPE;
    if (M == 0) return KQ_OK;
    if (!logits || !u || !tokens || !workspace) return KQ_ERR_NULL;
    const void *four[] = {logits, temperature, top_k, top_p, min_p, u, tokens, probs};
    for (const void *p : four)
        if (!aligned(p, 4)) return KQ_ERR_ALIGN;
    if (!aligned(workspace, 16)) return KQ_ERR_ALIGN;
    const SampleSpace s = sample_space(M, V);
    if (workspace_bytes < s.end) return KQ_ERR_SHAPE;
    if (device_check()) return KQ_ERR_DEVICE;
    uint8_t *ws = (uint8_t *)workspace;
    Sample a = {logits, temperature, top_p, min_p, u, top_k, tokens, probs, (u64 *)ws, (u32 *)(ws + s.near_n), (u64 *)(ws + s.near),
                (u64 *)(ws + s.hist), (uint16_t *)(ws + s.upto), (uint16_t *)(ws + s.order), ld, (int)V, s.chunks, 0};
    hipStream_t st = (hipStream_t)stream;
    for (; a.row0 < M; a.row0 += s.rows) {
        const int rows = std::min(M - a.row0, s.rows);
        hipLaunchKernelGGL(chunk_kernel, dim3((unsigned)a.chunks, (unsigned)rows), dim3(CHUNK_THREADS), 0, st, a);
        hipLaunchKernelGGL(row_kernel, dim3((unsigned)rows), dim3(ROW_THREADS), 0, st, a);
    }
    return kv::launched();
}

} // extern "C"
