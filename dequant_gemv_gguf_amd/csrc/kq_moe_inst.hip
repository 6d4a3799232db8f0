// kq_moe_inst.hip -- the experts' products of kqstep_moe for one block format,
// KQ_MOE_TYPE.
//
// Bound: HBM (a token's experts' weights, read once), for one token the chain of
// logits, choice, weights.  One work-group a compute unit, for one token and a
// tile of rows: a wave takes an expert and streams its rows through registers, two
// steps of them on the way at a time.  Each lane holds the activations of its unit
// of the rows (unit u on lane u % lanes_per_row of a lane group, see kq_impl.h) in
// registers: they are read once for all rows, and the loop reads no LDS for them.
// An expert that several tokens chose is read once per token, but their
// work-groups of one tile sit on one XCD and go through it side by side, so that
// its L2 serves the second read.
#include "kq_moe.h"

namespace kq {
namespace step {

constexpr int MOE_WAVES = 8, MOE_THREADS = 64 * MOE_WAVES;
constexpr int MOE_RESULTS = 8192;      // floats of LDS for the rows' sums

// How a call's rows lie on the grid: `waves` a work-group, `parts` of them a
// slot, `rows` of a matrix each; `tiles` work-groups a token.
struct Split {
    int lpr, waves, parts, rows, tiles;
    u32 magic;          // i * magic >> 16 = i / k
};

// XReg::load in two steps: the loads, and (once other loads are on their way) the
// sums, which wait for them.
template <int T> __device__ __forceinline__ void ask_unit(XReg<T> &xr, const float *x, int u) {
    typedef XReg<T> X;
    const float *p = x + unit_e0<T>(u);
#pragma unroll
    for (int i = 0; i < X::NV; ++i) xr.v[i] = *reinterpret_cast<const f4 *>(p + (X::RUNS32 ? 32 : 16) * (i / 4) + 4 * (i % 4));
}
template <int T> __device__ __forceinline__ void sum_unit(XReg<T> &xr) {
#pragma unroll
    for (int r = 0; r < XReg<T>::NS; ++r) xr.s[r] = sum16(xr.v[4 * r], xr.v[4 * r + 1], xr.v[4 * r + 2], xr.v[4 * r + 3]);
}
template <int T> __device__ __forceinline__ void ask_first(XReg<T> &xr, const float *x, int n, int lpr) {
    const int units = (n / Fmt<T>::QK) * Fmt<T>::UPB;
    ask_unit<T>(xr, x, min((int)threadIdx.x & (lpr - 1), units - 1));
}

// Sums of `count` rows (of row_bytes each, from the start of rs[m] + delta[m] on) of
// N matrices with the activations of unit u, added to (ADD) or put into
// out[m * count + row].  D units a lane are on their way, those of the N matrices
// in turn; `meanwhile` runs when the first ones are asked for.
template <int T, int N, int D, bool ADD, class Fn>
__device__ __forceinline__ void stream_rows(const rsrc_t (&rs)[N], const u32 (&delta)[N], u32 row_bytes, int count, int lpr, int u,
                                            bool in, XReg<T> &xr, float *out, Fn &&meanwhile) {
    typedef Fmt<T> F;
    typedef typename RawOf<T>::type Raw;
    constexpr int R = D / N;               // rows of a lane group a turn
    const int lane = threadIdx.x & 63, slot = lane & (lpr - 1), sh = __builtin_ctz(lpr), grp = lane >> sh, G = 64 >> sh;
    const int sub = u % F::UPB;
    const u32 boff = (u32)(u / F::UPB) * F::BYTES;
    Raw ring[D][1];
    // past the last row: zeros, and nothing is read
    auto issue = [&](int d, int row) {
        const int i = row + grp + G * (d / N);
        load_unit(ring[d][0], rs[d % N], in && i < count ? delta[d % N] + (u32)i * row_bytes + boff : OOB, sub);
    };
    const int idx = scatter_idx<D>(lane), row_of = grp + G * (idx / N);
#pragma unroll
    for (int d = 0; d < D; ++d) issue(d, 0);
    __builtin_amdgcn_sched_barrier(0);
    meanwhile();
    sum_unit<T>(xr);
    for (int row = 0; row < count; row += G * R) {
        float w[D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            __builtin_amdgcn_sched_barrier(0);
            float v[1][1];
            val_unit<1, 1>(ring[d], sub, xr, v);
            w[d] = in ? v[0][0] : 0.f;
            issue(d, row + G * R);
        }
        __builtin_amdgcn_sched_barrier(0);
        const float s = reduce_scatter<D>(w, lane, lpr);
        const int i = row + row_of;
        if (slot < D && i < count) {
            float *o = out + (idx % N) * count + i;
            *o = ADD ? *o + s : s;
        }
    }
}

// The same over whole rows of n activations at x; xr: those of the lane's first
// unit, asked for (its last one's afterwards: two sets would not fit the registers).
template <int T, int N, int D, class Fn>
__device__ __forceinline__ void row_sums(const uint8_t *const (&W)[N], int64_t row_bytes, int count, int n, int lpr, const float *x,
                                         XReg<T> &xr, float *out, Fn &&meanwhile) {
    const int slot = threadIdx.x & (lpr - 1), units = (n / Fmt<T>::QK) * Fmt<T>::UPB;
    rsrc_t rs[N];
    u32 delta[N];
#pragma unroll
    for (int m = 0; m < N; ++m) {
        const uintptr_t at = (uintptr_t)W[m];
        delta[m] = (u32)(at & 3u);
        rs[m] = make_rsrc((const void *)(at - delta[m]), delta[m] + (u32)(count * row_bytes));
    }
    stream_rows<T, N, D, false>(rs, delta, (u32)row_bytes, count, lpr, min(slot, units - 1), slot < units, xr, out, meanwhile);
    for (int u0 = lpr; u0 < units; u0 += lpr) {
        const int u = min(u0 + slot, units - 1);
        ask_unit<T>(xr, x, u);
        stream_rows<T, N, D, true>(rs, delta, (u32)row_bytes, count, lpr, u, u0 + slot < units, xr, out, meanwhile);
    }
}

// Keys order like the 64-bit values; NaN is the lowest, 1, and 0 an expert that is
// taken (or none).
__device__ __forceinline__ u64 order_of(double x) {
    const u64 b = __builtin_bit_cast(u64, x + 0.0);
    return x == x ? (b >> 63 ? ~b : b | (1ull << 63)) : 1ull;
}
__device__ __forceinline__ u32 wave_max_u32(u32 x) {
    x = max(x, (u32)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false));
    x = max(x, (u32)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false));
    x = max(x, (u32)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, false));
    x = max(x, (u32)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, false));
    const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max((u32)p[0], (u32)p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return max((u32)q[0], (u32)q[1]);
}
__device__ __forceinline__ double wave_max_d(double x) {
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) x = fmax(x, __shfl_xor(x, i));
    return x;
}

// The score of a logit is weight_of(l) / sum; a softmax's sum goes over all
// experts (by one wave), a sigmoid's is 1.
struct Scores { double max, sum; };
__device__ __forceinline__ double weight_of(const Moe &a, const Scores &s, double l) {
    return a.score == KQSTEP_SOFTMAX ? exp(l - s.max) : 1.0 / (1.0 + exp(-l));
}
__device__ __forceinline__ Scores scores_of(const Moe &a, const double *l) {
    Scores s = {0.0, 1.0};
    if (a.score != KQSTEP_SOFTMAX) return s;
    const int lane = threadIdx.x & 63;
    double max = -__builtin_inf(), sum = 0.0;
    for (int e = lane; e < a.E; e += 64) max = fmax(max, l[e]);
    s.max = wave_max_d(max);
    for (int e = lane; e < a.E; e += 64) sum += exp(l[e] - s.max);
    s.sum = sum_d<64>(sum);
    return s;
}

// The token's experts, by the whole work-group, into ids[0 .. k).
// PER 0: up to 256 experts.  An expert's place is the number of those that come
// before it; a thread counts them over a part of the experts.
// PER > 0: the first wave alone, a lane with PER neighbouring experts, takes k
// times the greatest of all that is left (its upper half first).  Counting takes
// E^2 steps over all threads, this one k of about 500 cycles whatever E: 0.6 and 1.7
// us for 8 of 128 experts.
constexpr int COUNTED = 256;
template <int PER, class Fn> __device__ __forceinline__ void choose(const Moe &a, const double *l, int E, int *ids, Fn &&meanwhile) {
    const int tid = threadIdx.x, lane = tid & 63;
    if constexpr (PER == 0) {
        __shared__ __align__(16) u64 keys[COUNTED];
        __shared__ int before[COUNTED];
        const int width = E <= 64 ? 64 : E <= 128 ? 128 : 256, e = tid & (width - 1), part = tid / width;
        const int parts = (int)blockDim.x / width, each = ((E + parts - 1) / parts + 1) & ~1;
        const double mine = l[min(e, E - 1)];
        __builtin_amdgcn_sched_barrier(0);
        meanwhile();
        __builtin_amdgcn_sched_barrier(0);
        if (part == 0) {
            u64 key = order_of(mine);
            if (__builtin_expect(a.bias != nullptr, 0)) {
                const Scores s = scores_of(a, l);
                key = order_of(weight_of(a, s, mine) / s.sum + (double)a.bias[min(e, E - 1)]);
            }
            keys[e] = e < E ? key : 0;
            before[e] = 0;
        }
        __syncthreads();
        // (a key of 0 comes before none; those behind E are 0)
        if (part < parts) {
            const u64 mine = keys[e];
            int n = 0;
            const int first = part * each, last = min(first + each, width);
            // (past the part: counted as none)
            for (int j0 = first; j0 < last; j0 += 16) {
                ulonglong2 two[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) two[i] = *(const ulonglong2 *)(keys + min(j0 + 2 * i, COUNTED - 2));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = j0 + 2 * i;
                    n += j < last && ((u64)two[i].x > mine || ((u64)two[i].x == mine && j < e));
                    n += j < last && ((u64)two[i].y > mine || ((u64)two[i].y == mine && j + 1 < e));
                }
            }
            if (parts > 1) atomicAdd(&before[e], n);
            else before[e] = n;
        }
        __syncthreads();
        if (tid < E && before[tid] < a.k) ids[before[tid]] = tid;
    } else {
        meanwhile();
        if (tid < 64) {
            const bool biased = a.bias != nullptr;
            Scores s = {0.0, 1.0};
            if (biased) s = scores_of(a, l);
            u64 key[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = lane * PER + i;
                key[i] = 0;
                if (e < E) key[i] = order_of(biased ? weight_of(a, s, l[e]) / s.sum + (double)a.bias[e] : l[e]);
            }
            for (int j = 0; j < a.k; ++j) {
                u64 best = key[0];
                int at = 0;
#pragma unroll
                for (int i = 1; i < PER; ++i)
                    if (key[i] > best) {
                        best = key[i];
                        at = i;
                    }
                const u32 hi = (u32)(best >> 32), lo = (u32)best;
                const u32 top = wave_max_u32(hi);
                u64 who = __ballot(hi == top);
                if (who & (who - 1)) {
                    const u32 low = wave_max_u32(hi == top ? lo : 0u);
                    who = __ballot(hi == top && lo == low);
                }
                const int winner = __builtin_ctzll(who);                 // the lowest lane has the lowest expert
                if (lane == winner) {
                    ids[j] = lane * PER + at;
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (i == at) key[i] = 0;
                }
            }
        }
    }
    __syncthreads();
}

// The weights of the token's experts (in `ids`), by one wave, lane i the i-th.
__device__ __forceinline__ float weights_of(const Moe &a, const double *l, const int32_t *ids) {
    const int lane = threadIdx.x & 63;
    const double mine = lane < a.k ? l[ids[lane]] : -__builtin_inf();
    Scores s = {0.0, 1.0};
    if (!a.renorm) s = scores_of(a, l);
    else if (a.score == KQSTEP_SOFTMAX) s.max = wave_max_d(mine);    // (the sum over all experts drops out)
    const double p = lane < a.k ? weight_of(a, s, mine) : 0.0;
    const double all = a.renorm ? sum_d<64>(p) : s.sum;
    return (float)(p / all * a.scale);
}

__device__ __forceinline__ float act_of(int act, float g) {
    if (act == KQSTEP_SILU) return g / (1.f + expf(-g));
    return 0.5f * g * (1.f + tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g)));
}

// Tile of a work-group (its token is blockIdx.y): those of one tile are 8 apart in
// the grid, on one XCD.
__device__ __forceinline__ int tile_of() { return blockIdx.z * 8 + blockIdx.x; }

// Orders a wave's LDS writes before its other lanes' reads.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int T, int D, int PER>
__global__ __launch_bounds__(MOE_THREADS) void gate_up_kernel(const double *logits, const float *xs, int E, int lpr, int hidden, int tiles,
                                                              const Moe a, const Split s) {
    __shared__ float results[MOE_RESULTS];
    __shared__ int ids[MOE_SLOTS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.y, tile = tile_of();
    if (tile >= tiles) return;
    XReg<T> xr;
    const float *x = xs;
    choose<PER>(a, logits + (int64_t)t * E, E, ids, [&] {
        x += t * a.ldx;
        ask_first<T>(xr, x, hidden, lpr);
    });
    if (tile == 0 && (int)threadIdx.x < a.k) a.ids[t * a.k + threadIdx.x] = ids[threadIdx.x];
    float *mine = results + wave * s.rows * 2;
    for (int i = wave; i < a.k * s.parts; i += s.waves) {
        const int part = (int)((u32)i * s.magic >> 16), j = i - part * a.k;
        const int first = (tile * s.parts + part) * s.rows, count = min(a.n_inner - first, s.rows);
        if (count <= 0) break;
        const int e = __builtin_amdgcn_readfirstlane(ids[j]);
        const int64_t base = ((int64_t)e * a.n_inner + first) * a.gate_bytes;
        const uint8_t *W[2] = {a.gate + base, a.up + base};
        if (i != wave) ask_first<T>(xr, x, a.hidden, s.lpr);
        row_sums<T, 2, D>(W, a.gate_bytes, count, a.hidden, s.lpr, x, xr, mine, [] {});
        wave_sync();
        float *out = a.inner + ((int64_t)t * a.k + j) * a.n_inner + first;
        for (int r = lane; r < count; r += 64) out[r] = act_of(a.act, mine[r]) * mine[count + r];
        wave_sync();
    }
}

// The slots' sums meet in LDS and are added in their order.
template <int T, int D>
__global__ __launch_bounds__(MOE_THREADS) void down_kernel(const int32_t *ids, const float *inner, int k, int n_inner, int lpr, u32 magic,
                                                           const Moe a, const Split s) {
    __shared__ float results[MOE_RESULTS];
    __shared__ float weights[MOE_SLOTS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.y, tile = tile_of();
    if (tile >= s.tiles) return;
    const int rows = s.rows * s.parts;
    for (int i = wave; i < a.k * s.parts; i += s.waves) {
        const int part = (int)((u32)i * magic >> 16), j = i - part * k;
        const int first = tile * rows + part * s.rows, count = min(a.hidden - first, s.rows);
        if (count <= 0) break;
        const float *x = inner + ((int64_t)t * k + j) * n_inner;
        XReg<T> xr;
        const int e = __builtin_amdgcn_readfirstlane(ids[t * k + j]);
        ask_first<T>(xr, x, n_inner, lpr);
        const uint8_t *W[1] = {a.down + ((int64_t)e * a.hidden + first) * a.down_bytes};
        row_sums<T, 1, D>(W, a.down_bytes, count, n_inner, lpr, x, xr, results + j * rows + part * s.rows, [&] {
            if (i == 0) {
                const float w = weights_of(a, a.logits + (int64_t)t * a.E, ids + t * k);
                if (lane < a.k) {
                    weights[lane] = w;
                    if (tile == 0 && a.weights) a.weights[t * a.k + lane] = w;
                }
            }
        });
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows; i += blockDim.x) {
        const int row = tile * rows + i;
        if (row >= a.hidden) break;
        float sum = a.add ? a.add[t * a.ldadd + row] : 0.f;
        for (int j = 0; j < a.k; ++j) sum = __builtin_fmaf(weights[j], results[j * rows + i], sum);
        a.y[t * a.ldy + row] = sum;
    }
}

// A work-group a compute unit (as many as fit beside each other make no
// difference to what is on its way), tiles of equal size.
static Split split_of(const Moe &a, int rows, int lpr, int results) {
    Split s;
    s.lpr = lpr;
    s.parts = a.k >= MOE_WAVES ? 1 : MOE_WAVES / a.k;
    s.waves = a.k > MOE_WAVES ? (a.k + 1) / 2 : a.k * s.parts;
    s.magic = (u32)((65536 + a.k - 1) / a.k);
    const int wgs = std::max(1, cu_count() / a.T);
    const int most = std::max(1, MOE_RESULTS / results);
    s.rows = std::min((rows + wgs * s.parts - 1) / (wgs * s.parts), most);
    s.tiles = (rows + s.rows * s.parts - 1) / (s.rows * s.parts);
    return s;
}

// Units a lane has on their way.
template <int T> constexpr int DEPTH() { return BIG_UNIT<T>() ? 2 : 4; }

template <int T, int PER> static void gate_up(const Moe &a, const Split &s, hipStream_t st) {
    hipLaunchKernelGGL((gate_up_kernel<T, DEPTH<T>(), PER>), dim3(8, (unsigned)a.T, (unsigned)((s.tiles + 7) / 8)), dim3(64 * s.waves), 0, st,
                       a.logits, a.x, a.E, s.lpr, a.hidden, s.tiles, a, s);
}
template <int T> int launch_gate_up(const Moe &a, hipStream_t st) {
    const int lpr = lanes_per_row(a.hidden / Fmt<T>::QK * Fmt<T>::UPB);
    const int waves = a.k > MOE_WAVES ? (a.k + 1) / 2 : a.k * std::max(1, MOE_WAVES / a.k);
    const Split s = split_of(a, a.n_inner, lpr, 2 * waves);
    if (a.E <= COUNTED) gate_up<T, 0>(a, s, st);
    else gate_up<T, MOE_EXPERTS / 64>(a, s, st);
    return kv::launched();
}
template <int T> int launch_down(const Moe &a, hipStream_t st) {
    const int lpr = lanes_per_row(a.n_inner / Fmt<T>::QK * Fmt<T>::UPB);
    const Split s = split_of(a, a.hidden, lpr, a.k * (a.k >= MOE_WAVES ? 1 : MOE_WAVES / a.k));
    hipLaunchKernelGGL((down_kernel<T, DEPTH<T>()>), dim3(8, (unsigned)a.T, (unsigned)((s.tiles + 7) / 8)), dim3(64 * s.waves), 0, st,
                       a.ids, a.inner, a.k, a.n_inner, s.lpr, s.magic, a, s);
    return kv::launched();
}

KQ_MOE_LAUNCHERS(template, KQ_MOE_TYPE)

} // namespace step
} // namespace kq
