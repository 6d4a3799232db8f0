// kq_moe_inst.hip -- the experts' products of kqstep_moe for one block format,
// KQ_MOE_TYPE.
//
// Bound: HBM (a token's experts' weights, read once).  A wave takes rows of one
// expert: each lane holds the activations of its unit of the row (unit u on lane
// u % lanes_per_row of a lane group, see kq_impl.h) in registers, asks for that
// unit of all its rows at once and keeps a partial sum a row, summed over the
// lanes at the end.  No LDS in that loop: an activation is read from the cache
// once for all of a wave's rows.
#include "kq_moe.h"

namespace kq {
namespace step {

constexpr int MOE_THREADS = 512, MOE_WG_WAVES = MOE_THREADS / 64;

// Sums over a lane group of rows first + grp + G * r, r < R, of N matrices at W
// (rows of row_bytes, `rows` of them), with the activations x.  Every lane of a
// group gets its group's sums.
template <int T, int N, int R>
__device__ __forceinline__ void row_sums(const uint8_t *const (&W)[N], int64_t row_bytes, int first, int rows,
                                         const float *x, int n, int lpr, float (&acc)[N * R]) {
    typedef Fmt<T> F;
    typedef typename RawOf<T>::type Raw;
    const int lane = threadIdx.x & 63, G = 64 / lpr, grp = lane / lpr, slot = lane - grp * lpr;
    const int units = (n / F::QK) * F::UPB;
    const int mine = min(rows - first, G * R);
    rsrc_t rs[N];
    u32 off[N * R];
#pragma unroll
    for (int m = 0; m < N; ++m) {
        const uintptr_t at = (uintptr_t)(W[m] + first * row_bytes);
        const u32 delta = (u32)(at & 3u);
        rs[m] = make_rsrc((const void *)(at - delta), delta + (u32)(mine * row_bytes));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = grp + G * r;
            off[m * R + r] = i < mine ? delta + (u32)(i * row_bytes) : OOB;
            acc[m * R + r] = 0.f;
        }
    }
    for (int u0 = 0; u0 < units; u0 += lpr) {
        const bool in = u0 + slot < units;
        const int u = in ? u0 + slot : 0, sub = u % F::UPB;
        const u32 boff = (u32)(u / F::UPB) * F::BYTES;
        Raw raw[N * R];
#pragma unroll
        for (int i = 0; i < N * R; ++i) load_unit(raw[i], rs[i / R], in ? off[i] + boff : OOB, sub);
        XReg<T> xr;
        xr.load(x, unit_e0<T>(u));
        float v[N * R][1];
        val_unit<1, N * R>(raw, sub, xr, v);
#pragma unroll
        for (int i = 0; i < N * R; ++i) acc[i] += in ? v[i][0] : 0.f;
    }
    group_sum_n<N * R>(acc, lpr);
}

// The token's experts, by the first wave: k times the largest logit (with a
// bias: score) that is left.  Keys order like the 64-bit values; NaN is the lowest,
// 1, and 0 an expert that is taken.
__device__ __forceinline__ u64 order_of(double x) {
    const u64 b = __builtin_bit_cast(u64, x + 0.0);
    return x == x ? (b >> 63 ? ~b : b | (1ull << 63)) : 1ull;
}
__device__ __forceinline__ double score_of(const Moe &a, double l, double max) {
    return a.score == KQSTEP_SOFTMAX ? exp(l - max) : 1.0 / (1.0 + exp(-l));
}

__device__ __forceinline__ void choose(const Moe &a, int t, int *ids, float *weights) {
    __shared__ u64 left[MOE_EXPERTS];
    const int lane = threadIdx.x;
    const double *l = a.logits + (int64_t)t * a.E;
    double max = -__builtin_inf();
    for (int e = lane; e < a.E; e += 64) max = fmax(max, l[e]);
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) max = fmax(max, __shfl_xor(max, i));
    double sum = 0.0;
    if (a.score == KQSTEP_SOFTMAX) {
        for (int e = lane; e < a.E; e += 64) sum += exp(l[e] - max);
        sum = sum_d<64>(sum);
    } else {
        sum = 1.0;
    }
    for (int e = lane; e < a.E; e += 64)
        left[e] = order_of(a.bias ? score_of(a, l[e], max) / sum + (double)a.bias[e] : l[e]);
    double p = 0.0;
    int chosen = 0;
    for (int j = 0; j < a.k; ++j) {
        u64 best = 0;
        int who = -1;
        for (int e = lane; e < a.E; e += 64)
            if (left[e] > best) {
                best = left[e];
                who = e;
            }
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) {
            const u64 o = (u64)__shfl_xor((long long)best, i);
            const int w = __shfl_xor(who, i);
            if (o > best || (o == best && (u32)w < (u32)who)) {
                best = o;
                who = w;
            }
        }
        if ((who & 63) == lane) left[who] = 0;
        if (lane == j) chosen = who;
    }
    const bool one = lane < a.k;
    if (one) p = score_of(a, l[chosen], max) / sum;
    const double all = sum_d<64>(p);
    if (one) {
        ids[lane] = chosen;
        weights[lane] = (float)(a.renorm ? p / all * a.scale : p * a.scale);
    }
}

__device__ __forceinline__ float act_of(int act, float g) {
    if (act == KQSTEP_SILU) return g / (1.f + expf(-g));
    return 0.5f * g * (1.f + tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g)));
}

constexpr int GATE_R = 2, DOWN_R = 2;

// Work-group (tile of inner rows, token): its waves take (slot, part of the
// tile) in turn.
template <int T>
__global__ __launch_bounds__(MOE_THREADS) void gate_up_kernel(const Moe a, int lpr, int parts) {
    __shared__ int ids[MOE_SLOTS];
    __shared__ float weights[MOE_SLOTS];
    const int t = blockIdx.y, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (wave == 0) {
        choose(a, t, ids, weights);
        if (blockIdx.x == 0 && lane < a.k) {
            a.ids[t * a.k + lane] = ids[lane];
            a.weights[t * a.k + lane] = weights[lane];
        }
    }
    __syncthreads();
    const int G = 64 / lpr, grp = lane / lpr;
    for (int i = wave; i < a.k * parts; i += MOE_WG_WAVES) {
        const int part = i / a.k, j = i - part * a.k;
        const int first = (blockIdx.x * parts + part) * G * GATE_R;
        if (first >= a.n_inner) break;
        const int e = __builtin_amdgcn_readfirstlane(ids[j]);
        const int64_t base = (int64_t)e * a.n_inner * a.gate_bytes;
        const uint8_t *W[2] = {a.gate + base, a.up + base};
        float v[2 * GATE_R];
        row_sums<T, 2, GATE_R>(W, a.gate_bytes, first, a.n_inner, a.x + t * a.ldx, a.hidden, lpr, v);
        float *out = a.inner + ((int64_t)t * a.k + j) * a.n_inner;
#pragma unroll
        for (int r = 0; r < GATE_R; ++r) {
            const int row = first + grp + G * r;
            if (lane - grp * lpr == 0 && row < a.n_inner) out[row] = act_of(a.act, v[r]) * v[GATE_R + r];
        }
    }
}

// Work-group (tile of hidden rows, token): as above; the slots' sums meet in
// LDS and are added in their order.
template <int T>
__global__ __launch_bounds__(MOE_THREADS) void down_kernel(const Moe a, int lpr, int parts) {
    __shared__ float sums[MOE_SLOTS * 4 * DOWN_R];       // [slot][row]: k * parts <= 16
    const int t = blockIdx.y, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int G = 64 / lpr, grp = lane / lpr, tile = parts * G * DOWN_R;
    for (int i = wave; i < a.k * parts; i += MOE_WG_WAVES) {
        const int part = i / a.k, j = i - part * a.k;
        const int first = blockIdx.x * tile + part * G * DOWN_R;
        if (first >= a.hidden) break;
        const int e = __builtin_amdgcn_readfirstlane(a.ids[t * a.k + j]);
        const uint8_t *W[1] = {a.down + (int64_t)e * a.hidden * a.down_bytes};
        float v[DOWN_R];
        row_sums<T, 1, DOWN_R>(W, a.down_bytes, first, a.hidden, a.inner + ((int64_t)t * a.k + j) * a.n_inner, a.n_inner,
                               lpr, v);
#pragma unroll
        for (int r = 0; r < DOWN_R; ++r)
            if (lane - grp * lpr == 0) sums[j * tile + part * G * DOWN_R + grp + G * r] = v[r];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tile; i += MOE_THREADS) {
        const int row = blockIdx.x * tile + i;
        if (row >= a.hidden) break;
        float s = a.add ? a.add[t * a.ldadd + row] : 0.f;
        for (int j = 0; j < a.k; ++j) s = __builtin_fmaf(a.weights[t * a.k + j], sums[j * tile + i], s);
        a.y[t * a.ldy + row] = s;
    }
}

// Parts of a tile, so that every wave has one: k * parts <= 16.
static int parts_of(int k) { return k >= MOE_WG_WAVES ? 1 : MOE_WG_WAVES / k; }

template <int T> int launch_gate_up(const Moe &a, hipStream_t st) {
    const int lpr = lanes_per_row(a.hidden / Fmt<T>::QK * Fmt<T>::UPB), parts = parts_of(a.k);
    const int tile = 64 / lpr * GATE_R * parts;
    hipLaunchKernelGGL(gate_up_kernel<T>, dim3((unsigned)((a.n_inner + tile - 1) / tile), (unsigned)a.T), dim3(MOE_THREADS), 0, st,
                       a, lpr, parts);
    return kv::launched();
}
template <int T> int launch_down(const Moe &a, hipStream_t st) {
    const int lpr = lanes_per_row(a.n_inner / Fmt<T>::QK * Fmt<T>::UPB), parts = parts_of(a.k);
    const int tile = 64 / lpr * DOWN_R * parts;
    hipLaunchKernelGGL(down_kernel<T>, dim3((unsigned)((a.hidden + tile - 1) / tile), (unsigned)a.T), dim3(MOE_THREADS), 0, st, a,
                       lpr, parts);
    return kv::launched();
}

KQ_MOE_LAUNCHERS(template, KQ_MOE_TYPE)

} // namespace step
} // namespace kq
