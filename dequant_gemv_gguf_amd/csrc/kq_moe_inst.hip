// kq_moe_inst.hip -- the experts' products of kqstep_moe for one block format,
// KQ_MOE_TYPE.
//
// Bound: HBM (a token's experts' weights, read once) and, from three tokens on, the
// vector units' work on them (8 of 128 experts of 2048 x 768, Q4_K and Q6_K, one token:
// 16 us; eight tokens 47, 3.4 TB/s of the distinct experts' bytes; three tokens, 6 of 160
// of 5120 x 1536, Q5_K and Q4_K: 84, 3.1 TB/s, the vector units busy half the time with
// three waves a SIMD); for one token the chain of logits, choice, weights.
// A work-group takes one token and a tile of rows, a wave one expert's rows of the
// tile: it streams them through registers.  The activations are put into LDS once for
// the work-group (asked for by every wave from the cache they took 3300 cycles before
// its first weights) and from there into registers, those of a lane's unit (unit u on
// lane u % lanes_per_row of a lane group, see kq_impl.h), while the first weights are
// on their way: the loop itself reads no LDS.
// An expert that several tokens chose is read once per token, but their
// work-groups of one tile sit on one XCD and go through it side by side, so that
// its L2 serves the second read; it is unpacked for each.
#include "kq_moe.h"

namespace kq {
namespace step {

// Waves of a work-group, at most, and of a compute unit: as many as the kernel's
// registers let on its SIMDs.
constexpr int MOE_WAVES = 8;
template <int T> constexpr int GATE_RESIDENT() { return BIG_UNIT<T>() || T == T_Q2_K ? 12 : 16; }
template <int T> constexpr int DOWN_RESIDENT() { return BIG_UNIT<T>() ? 12 : 16; }
// Units of a lane on their way in a wave, of all formats.  (Two in the down kernel took a
// quarter of the waves' registers and were slower: eight tokens 49.7 -> 48.3 us with one.
// Four in gate and up: five tokens of Q8_0 16.8 -> 19.9, four 48.7 -> 50.2, six of Q2_K
// 48.9 -> 53.6.)
constexpr int GATE_DEPTH = 2, DOWN_DEPTH = 1;
constexpr int MOE_LDS = 54 * 1024 / 4;         // floats of LDS that a launch asks for, at most (64 KB with the kernels' own)
constexpr int MOE_RESULTS = 2048;              // of them for the rows' sums

// How a call's rows lie on the grid: `waves` a work-group, `parts` of them a
// slot, `rows` of a matrix each; `tiles` work-groups a token.
struct Split {
    int lpr, waves, parts, rows, tiles;
    u32 magic;          // i * magic >> 16 = i / k
    u32 row_magic;      // i * row_magic >> 32 = i / (a staged row's length)
    int staged;         // whether the activations go through LDS
};

// XReg::load in two steps, for rows that do not fit LDS: the loads, and the sums,
// which wait for them.
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

// A row of n activations into LDS as stage_x leaves them, 4 a thread: asked for, and put.
constexpr int ASK = 4;
__device__ __forceinline__ void ask_row(f4 (&v)[ASK], const float *x, int n, int from, int threads) {
#pragma unroll
    for (int i = 0; i < ASK; ++i) {
        const int e = 4 * (from + (int)threadIdx.x + i * threads);
        v[i] = *reinterpret_cast<const f4 *>(x + (e < n ? e : 0));
    }
}
__device__ __forceinline__ void put_row(const f4 (&v)[ASK], float *xs, float *ss, int n, int from, int threads) {
#pragma unroll
    for (int i = 0; i < ASK; ++i) {
        const int e = 4 * (from + (int)threadIdx.x + i * threads);
        // (n is a multiple of 32: the four lanes of 16 activations are here together)
        float s = (v[i].x + v[i].y) + (v[i].z + v[i].w);
        s = dpp_add(s, 0);
        s = dpp_add(s, 1);
        if (e < n) {
            *reinterpret_cast<f4 *>(xs + xpad(e)) = v[i];
            if ((e & 15) == 0) ss[e >> 4] = s;
        }
    }
}
__device__ __forceinline__ void stage_row(float *xs, float *ss, const float *x, int n, int from, int threads) {
    for (; 4 * from < n; from += ASK * threads) {
        f4 v[ASK];
        ask_row(v, x, n, from, threads);
        put_row(v, xs, ss, n, from, threads);
    }
}

// The activations of a lane's unit: from LDS (xs: a staged row of n), or from x.
struct Activations {
    const float *xs, *x;
    int n;
    template <int T> __device__ __forceinline__ void unit(XReg<T> &xr, int u) const {
        if (xs) {
            const int e0 = unit_e0<T>(u);
            xreg_from_lds<T>(xr, XLds{xs, xs + x_stride(n), 0, 0, xpad(e0), e0 >> 4, sum_run_stride<T>()});
        } else {
            ask_unit<T>(xr, x, u);
            sum_unit<T>(xr);
        }
    }
};

// Sums of `count` rows (of row_bytes each, from the start of rs[m] + delta[m] on) of
// N matrices with the activations of units u0 + the lane's, added to (ADD) or put into
// out[m * count + row].
template <int T, int N, int DEPTH, bool ADD>
__device__ __forceinline__ void stream_rows(const rsrc_t (&rs)[N], const u32 (&delta)[N], u32 row_bytes, int count, int lpr, int u0,
                                            const Activations &x, float *out) {
    typedef Fmt<T> F;
    typedef typename RawOf<T>::type Raw;
    constexpr int R = DEPTH / N;           // rows of a lane group a turn
    const int lane = threadIdx.x & 63, slot = lane & (lpr - 1), sh = __builtin_ctz(lpr), grp = lane >> sh, G = 64 >> sh;
    const int units = (x.n / F::QK) * F::UPB;
    const bool in = u0 + slot < units;
    const int u = in ? u0 + slot : 0, sub = u % F::UPB;
    const u32 boff = (u32)(u / F::UPB) * F::BYTES;
    Raw ring[DEPTH][1];
    // past the last row: zeros, and nothing is read
    auto issue = [&](int d, int row) {
        const int i = row + grp + G * (d / N);
        load_unit(ring[d][0], rs[d % N], in && i < count ? delta[d % N] + (u32)i * row_bytes + boff : OOB, sub);
    };
    const int idx = scatter_idx<DEPTH>(lane), row_of = grp + G * (idx / N);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) issue(d, 0);
    __builtin_amdgcn_sched_barrier(0);
    XReg<T> xr;
    x.unit<T>(xr, u);
    for (int row = 0; row < count; row += G * R) {
        float w[DEPTH];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            __builtin_amdgcn_sched_barrier(0);
            float v[1][1];
            val_unit<1, 1>(ring[d], sub, xr, v);
            w[d] = in ? v[0][0] : 0.f;
            issue(d, row + G * R);
        }
        __builtin_amdgcn_sched_barrier(0);
        const float s = reduce_scatter<DEPTH>(w, lane, lpr);
        const int i = row + row_of;
        if (slot < DEPTH && i < count) {
            float *o = out + (idx % N) * count + i;
            *o = ADD ? *o + s : s;
        }
    }
}

// The same over whole rows.
template <int T, int N, int DEPTH>
__device__ __forceinline__ void row_sums(const uint8_t *const (&W)[N], int64_t row_bytes, int count, int lpr, const Activations &x,
                                         float *out) {
    const int units = (x.n / Fmt<T>::QK) * Fmt<T>::UPB;
    rsrc_t rs[N];
    u32 delta[N];
#pragma unroll
    for (int m = 0; m < N; ++m) {
        const uintptr_t at = (uintptr_t)W[m];
        delta[m] = (u32)(at & 3u);
        rs[m] = make_rsrc((const void *)(at - delta[m]), delta[m] + (u32)(count * row_bytes));
    }
    stream_rows<T, N, DEPTH, false>(rs, delta, (u32)row_bytes, count, lpr, 0, x, out);
    for (int u0 = lpr; u0 < units; u0 += lpr) stream_rows<T, N, DEPTH, true>(rs, delta, (u32)row_bytes, count, lpr, u0, x, out);
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

// The token's experts, by the whole work-group (`waves` of them), into ids[0 .. k);
// `meanwhile` runs while the logits are on their way.
// MANY false: up to 256 experts, which are no more than threads.  An expert's place is the
// number of those with greater keys; a thread counts them over a part of the experts.
// Equal keys share a place, which the lower expert has, and leave one empty behind it:
// only then are those of the same key in front of each counted too.  (With the expert's
// number in a key's low bits there are none, but logits that differ by less than 2^-44 of
// their size counted as the same.)
// MANY: the first wave alone, a lane with every 64th expert, takes k times the
// greatest of all that is left (its upper half first).  Counting takes E^2 steps over
// all threads, this one k of about 500 cycles whatever E.
constexpr int COUNTED = 256;
template <bool MANY, class Fn> __device__ __forceinline__ void choose(const Moe &a, const double *l, int E, int waves, int *ids, Fn &&meanwhile) {
    const int tid = threadIdx.x, lane = tid & 63;
    if constexpr (!MANY) {
        __shared__ __align__(16) u64 keys[COUNTED];
        __shared__ int before[COUNTED];
        const int sh = E <= 64 ? 6 : E <= 128 ? 7 : 8, width = 1 << sh, e = tid & (width - 1), part = tid >> sh;
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
            if (e < MOE_SLOTS) ids[e] = MOE_EXPERTS;
        }
        __syncthreads();
        // (keys past the last expert are 0; the parts past `width` have none)
        const int parts = waves * 64 >> sh, each = width / (parts >= 4 ? 4 : parts >= 2 ? 2 : 1);
        if (part * each < width) {
            const u64 mine = keys[e];
            int n = 0;
            for (int j0 = part * each; j0 < (part + 1) * each && j0 < E; j0 += 16) {
                ulonglong2 two[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) two[i] = *(const ulonglong2 *)(keys + j0 + 2 * i);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    n += (u64)two[i].x > mine;
                    n += (u64)two[i].y > mine;
                }
            }
            if (each < width) atomicAdd(&before[e], n);
            else before[e] = n;
        }
        __syncthreads();
        if (tid < E && before[tid] < a.k) atomicMin(&ids[before[tid]], tid);
        __syncthreads();
        if (__builtin_expect(__ballot(lane < a.k && ids[lane < a.k ? lane : 0] == MOE_EXPERTS) != 0, 0)) {
            __syncthreads();
            if (tid < E && before[tid] < a.k) {
                int place = before[tid];
                for (int j = 0; j < tid; ++j) place += keys[j] == keys[tid];
                if (place < a.k) ids[place] = tid;
            }
            __syncthreads();
        }
    } else {
        __shared__ u64 left[MOE_EXPERTS];
        meanwhile();
        if (tid < 64) {
            Scores s = {0.0, 1.0};
            if (a.bias) s = scores_of(a, l);
            u64 best = 0;
            int who = 0;
            for (int e = lane; e < E; e += 64) {
                const u64 key = order_of(a.bias ? weight_of(a, s, l[e]) / s.sum + (double)a.bias[e] : l[e]);
                left[e] = key;
                if (key > best) {
                    best = key;
                    who = e;
                }
            }
            for (int j = 0; j < a.k; ++j) {
                const u32 hi = (u32)(best >> 32), lo = (u32)best;
                const u32 top = wave_max_u32(hi), low = wave_max_u32(hi == top ? lo : 0u);
                // the lowest of those that have it
                const u32 first = ~wave_max_u32(hi == top && lo == low ? ~(u32)who : 0u);
                if ((u32)who == first && best) {
                    ids[j] = who;
                    left[who] = 0;
                    best = 0;
                    for (int e = lane; e < E; e += 64)
                        if (left[e] > best) {
                            best = left[e];
                            who = e;
                        }
                }
            }
        }
        __syncthreads();
    }
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

extern __shared__ __align__(16) float moe_lds[];

// The work-group behind a token's last tile computes the weights of its experts.
template <int T, bool MANY>
__global__ __launch_bounds__(64 * MOE_WAVES) void gate_up_kernel(const double *logits, const float *xs, int64_t ldx, int E, int hidden,
                                                                     const Moe a, const Split s) {
    __shared__ int ids[MOE_SLOTS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.y, tile = tile_of();
    const float *x = xs + t * ldx;
    logits += (int64_t)t * E;
    const Activations act = {s.staged ? moe_lds : nullptr, x, hidden};
    choose<MANY>(a, logits, E, s.waves, ids, [&] {
        if (s.staged && tile < s.tiles) stage_row(moe_lds, moe_lds + x_stride(hidden), x, hidden, 0, 64 * s.waves);
    });
    if (tile >= s.tiles) {
        if (tile == s.tiles && wave == 0) {
            const float w = weights_of(a, logits, ids);
            if (lane < a.k) {
                a.ids[t * a.k + lane] = ids[lane];
                a.weights[t * a.k + lane] = w;
            }
        }
        return;
    }
    float *mine = moe_lds + (s.staged ? x_stride(hidden) + s_stride(hidden) : 0) + wave * s.rows * 2;
    for (int i = wave; i < a.k * s.parts; i += s.waves) {
        const int part = (int)((u32)i * s.magic >> 16), j = i - part * a.k;
        const int first = (tile * s.parts + part) * s.rows, count = min(a.n_inner - first, s.rows);
        if (count <= 0) break;
        const int e = __builtin_amdgcn_readfirstlane(ids[j]);
        const int64_t base = ((int64_t)e * a.n_inner + first) * a.gate_bytes;
        const uint8_t *W[2] = {a.gate + base, a.up + base};
        row_sums<T, 2, GATE_DEPTH>(W, a.gate_bytes, count, s.lpr, act, mine);
        wave_sync();
        float *out = a.inner + ((int64_t)t * a.k + j) * a.n_inner + first;
        for (int r = lane; r < count; r += 64) out[r] = act_of(a.act, mine[r]) * mine[count + r];
        wave_sync();
    }
}

// The slots' sums meet in LDS and are added in their order.
template <int T>
__global__ __launch_bounds__(64 * MOE_WAVES) void down_kernel(const int32_t *ids, const float *inner, int k, int n_inner, int waves, int staged,
                                                                  const Moe a, const Split s) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.y, tile = tile_of();
    if (tile >= s.tiles) return;
    inner += (int64_t)t * k * n_inner;
    ids += t * k;
    const int stride = x_stride(n_inner) + s_stride(n_inner);
    // the slots' rows (each a multiple of 32 long) as they lie behind each other
    f4 v[ASK];
    if (staged) ask_row(v, inner, k * n_inner, 0, 64 * waves);
    // the wave's first expert, whose number is on its way as well
    const int first_id = ids[wave < k ? wave : (int)((u32)wave % (u32)k)];
    if (staged) {
        const int threads = 64 * waves;
        for (int from = 0;;) {
#pragma unroll
            for (int i = 0; i < ASK; ++i) {
                const int e = 4 * (from + (int)threadIdx.x + i * threads), j = (int)__umulhi((u32)e, s.row_magic), at = e - j * n_inner;
                float sum = (v[i].x + v[i].y) + (v[i].z + v[i].w);
                sum = dpp_add(sum, 0);
                sum = dpp_add(sum, 1);
                if (j < k) {
                    float *xs = moe_lds + j * stride;
                    *reinterpret_cast<f4 *>(xs + xpad(at)) = v[i];
                    if ((at & 15) == 0) xs[x_stride(n_inner) + (at >> 4)] = sum;
                }
            }
            from += ASK * threads;
            if (4 * from >= k * n_inner) break;
            ask_row(v, inner, k * n_inner, from, threads);
        }
        __syncthreads();
    }
    float *results = moe_lds + (staged ? k * stride : 0);
    const int rows = s.rows * s.parts;
    for (int i = wave; i < k * s.parts; i += waves) {
        const int part = (int)((u32)i * s.magic >> 16), j = i - part * k;
        const int first = tile * rows + part * s.rows, count = min(a.hidden - first, s.rows);
        if (count <= 0) break;
        const int e = __builtin_amdgcn_readfirstlane(i == wave ? first_id : ids[j]);
        const uint8_t *W[1] = {a.down + ((int64_t)e * a.hidden + first) * a.down_bytes};
        const Activations x = {staged ? moe_lds + j * stride : nullptr, inner + (int64_t)j * n_inner, n_inner};
        row_sums<T, 1, DOWN_DEPTH>(W, a.down_bytes, count, s.lpr, x, results + j * rows + part * s.rows);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows; i += 64 * waves) {
        const int row = tile * rows + i;
        if (row >= a.hidden) break;
        float sum = a.add ? a.add[t * a.ldadd + row] : 0.f;
        for (int j = 0; j < k; ++j) sum = __builtin_fmaf(a.weights[t * k + j], results[j * rows + i], sum);
        a.y[t * a.ldy + row] = sum;
    }
}

// Tiles of equal size for all the work-groups that run at once; `matrices` of `rows`
// rows of n weights, `units` units, `floats` of LDS for the activations of a work-group.
static Split split_of(const Moe &a, int depth, int resident, int rows, int matrices, int units, int n, int64_t floats, int spare) {
    Split s;
    s.parts = a.k >= MOE_WAVES ? 1 : MOE_WAVES / a.k;
    // (waves of a work-group take the slots in equal rounds)
    const int rounds = (a.k * s.parts + MOE_WAVES - 1) / MOE_WAVES;
    s.waves = (a.k * s.parts + rounds - 1) / rounds;
    s.magic = (u32)((65536 + a.k - 1) / a.k);
    // (exact below 2^32 / n: the rows staged have fewer than 2^14 activations in all)
    s.row_magic = (u32)(((1ull << 32) + n - 1) / n);
    const int slots = matrices == 2 ? s.waves : a.k * s.parts;          // that hold results at once
    const int most = MOE_RESULTS / (matrices * slots);
    auto rows_of = [&](int T) {
        const int wgs = std::max(1, resident / s.waves * cu_count() / T - spare);
        return std::min((rows + wgs * s.parts - 1) / (wgs * s.parts), most);
    };
    s.rows = rows_of(a.T);
    s.tiles = (rows + s.rows * s.parts - 1) / (s.rows * s.parts);
    s.staged = floats + MOE_RESULTS <= MOE_LDS;
    // Lanes of a row: those with which a wave's rows take the fewest turns, where
    // another part of a row costs more than a unit for its activations (three tokens of 5120 x 1536, rows of 80
    // units: three parts of 32 lanes 85 us, five of 16 lanes 88).  (As
    // one token's call has them: a row's sum, whose order follows from it, is the same
    // in every call.)
    const int one = rows_of(1);
    int best = 0;
    for (int lpr = 16; lpr <= 64; lpr *= 2) {
        const int stripes = (units + lpr - 1) / lpr, turns = (one * matrices * lpr + 64 * depth - 1) / (64 * depth) * depth;
        const int cost = stripes * (3 * turns + 4);
        if (!best || cost < best) {
            best = cost;
            s.lpr = lpr;
        }
    }
    return s;
}

static dim3 moe_grid(const Moe &a, int tiles) { return dim3(8, (unsigned)a.T, (unsigned)((tiles + 7) / 8)); }

template <int T, bool MANY> static void gate_up(const Moe &a, const Split &s, size_t lds, hipStream_t st) {
    hipLaunchKernelGGL((gate_up_kernel<T, MANY>), moe_grid(a, s.tiles + 1), dim3(64 * s.waves), lds, st, a.logits, a.x, a.ldx, a.E, a.hidden, a, s);
}
template <int T> int launch_gate_up(const Moe &a, hipStream_t st) {
    const int64_t floats = x_stride(a.hidden) + s_stride(a.hidden);
    const Split s = split_of(a, GATE_DEPTH, GATE_RESIDENT<T>(), a.n_inner, 2, a.hidden / Fmt<T>::QK * Fmt<T>::UPB, a.hidden, floats, 1);
    const size_t lds = sizeof(float) * (size_t)((s.staged ? floats : 0) + 2 * s.rows * s.waves);
    if (a.E <= COUNTED) gate_up<T, false>(a, s, lds, st);      // (s.waves is 5 or more: a thread an expert)
    else gate_up<T, true>(a, s, lds, st);
    return kv::launched();
}
template <int T> int launch_down(const Moe &a, hipStream_t st) {
    const int64_t floats = (int64_t)a.k * (x_stride(a.n_inner) + s_stride(a.n_inner));
    const Split s = split_of(a, DOWN_DEPTH, DOWN_RESIDENT<T>(), a.hidden, 1, a.n_inner / Fmt<T>::QK * Fmt<T>::UPB, a.n_inner, floats, 0);
    const size_t lds = sizeof(float) * (size_t)((s.staged ? floats : 0) + s.rows * s.parts * a.k);
    hipLaunchKernelGGL(down_kernel<T>, moe_grid(a, s.tiles), dim3(64 * s.waves), lds, st, a.ids, a.inner, a.k, a.n_inner, s.waves, s.staged, a, s);
    return kv::launched();
}

KQ_MOE_LAUNCHERS(template, KQ_MOE_TYPE)

} // namespace step
} // namespace kq
