// kq_sample.hip -- a token for each row of logits (include/kqstep.h).
//
// Everything that the filters leave is a leading part of the tokens in the order
// of (logit descending, index ascending), so a filter is a place in that order:
// a logit's key (its bits, made to order like integers) and how many of the
// tokens with that very key stay.  A place is found digit by digit of the key,
// from the counts (top_k) or the summed weights (top_p) of the tokens that share
// its digits so far.  Weights are 64-bit integers, multiples of 2^-42: sums of
// them are exact, so that it does not matter in which order LDS atomics add them.
#include "kq_step.h"

#include <cmath>

namespace kq {
namespace step {

constexpr int ROW_THREADS = 1024, ROW_WAVES = ROW_THREADS / 64;
constexpr int CHUNK = 4096;                       // tokens whose kept weight is summed apart
constexpr int MAX_V = 1 << 20, MAX_CHUNKS = MAX_V / CHUNK;
constexpr double ONE = 4398046511104.0;           // 2^42, the weight of the largest logit

struct Sample {
    const float *logits, *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *tokens;
    float *probs;
    int64_t ld;
    int V;
};

// The key of a logit: 0 for what is never taken.  (+ 0: the zeros are equal.)
__device__ __forceinline__ u32 key_of(float l) {
    const u32 b = __builtin_bit_cast(u32, l + 0.f);
    return l > -__builtin_inff() ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float logit_of(u32 key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Weight of a key in a row whose largest key is `top`.
struct Weigh {
    u32 top;
    double max, t;
    __device__ __forceinline__ u64 operator()(u32 key) const {
        if (key == top) return (u64)ONE;
        const double d = (double)logit_of(key) - max;
        return key && d > -__builtin_inf() ? (u64)rint(exp(d / t) * ONE) : 0;
    }
};

__device__ __forceinline__ u64 wave_max(u64 x) {
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
        const u64 o = (u64)__shfl_xor((long long)x, i);
        x = o > x ? o : x;
    }
    return x;
}
__device__ __forceinline__ u64 wave_scan(u64 x, int lane) {      // inclusive
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
        const u64 o = (u64)__shfl_up((long long)x, i);
        if (lane >= i) x += o;
    }
    return x;
}

// A place in the order: tokens with a greater key, and the first `ties` of those
// with this one.
struct Place { u32 key, ties; };

// One row, a work-group: each step goes over the whole row.
__global__ __launch_bounds__(ROW_THREADS) void sample_kernel(const Sample a) {
    __shared__ u64 hist[256], chunk_weight[MAX_CHUNKS], waves[ROW_WAVES];
    __shared__ u32 chunk_ties[MAX_CHUNKS];
    __shared__ u64 found[3];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float *l = a.logits + row * a.ld;
    const float t = a.temperature ? a.temperature[row] : 1.f;
    // the first token of the order
    u64 best = 0;
    for (int i = tid; i < a.V; i += ROW_THREADS) {
        const u64 x = (u64)key_of(l[i]) << 32 | (u32)~i;
        best = x > best ? x : best;
    }
    best = wave_max(best);
    if (lane == 0) waves[wave] = best;
    __syncthreads();
    best = wave_max(waves[lane & (ROW_WAVES - 1)]);
    const u32 top = (u32)(best >> 32);
    const int first = (int)~(u32)best;
    if (!top || !(t > 0.f)) {
        if (tid == 0) {
            a.tokens[row] = top ? first : -1;
            if (a.probs) a.probs[row] = top ? 1.f : 0.f;
        }
        return;
    }
    const Weigh weigh = {top, (double)logit_of(top), (double)t};

    // The shortest leading part of `in` of which `by` (1: tokens, 2: weights)
    // sums to at least `want`, and its sum of weights.
    auto cut = [&](Place in, bool weights, u64 want, Place *out, u64 *weight) {
        u32 prefix = 0;
        u64 before = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int i = tid; i < a.V; i += ROW_THREADS) {
                const u32 key = key_of(l[i]);
                if (key <= in.key || (shift < 24 && key >> (shift + 8) != prefix)) continue;
                atomicAdd((unsigned long long *)&hist[(key >> shift) & 255], weights ? weigh(key) : 1ull);
            }
            __syncthreads();
            if (tid < 64) {
                // 4 digits a lane, descending
                u64 d[4], s = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32 digit = 255 - (4 * lane + i);
                    d[i] = hist[digit];
                    if (in.ties && (shift == 24 || in.key >> (shift + 8) == prefix) && ((in.key >> shift) & 255) == digit)
                        d[i] += in.ties * (weights ? weigh(in.key) : 1ull);
                    s += d[i];
                }
                const u64 upto = wave_scan(s, lane);
                const u64 reach = __ballot(before + upto >= want);
                // (the sum over all digits reaches `want`, unless it is 0)
                const int at = reach ? __builtin_ctzll(reach) : 63;
                if (lane == at) {
                    u64 sum = before + upto - s;
                    int i = 0;
                    for (; i < 3 && sum + d[i] < want; ++i) sum += d[i];
                    found[0] = (u64)(255 - (4 * lane + i));
                    found[1] = sum;
                }
            }
            __syncthreads();
            prefix = prefix << 8 | (u32)found[0];
            before = found[1];
        }
        // tokens of this key: one tokens's worth after the other
        const u64 each = weights ? weigh(prefix) : 1;
        const u64 need = want > before ? want - before : 0;
        u64 n = each ? (need + each - 1) / each : 0;
        n = n ? n : 1;
        if (prefix == in.key && n > in.ties) n = in.ties;
        out->key = prefix;
        out->ties = (u32)n;
        *weight = before + n * each;
        __syncthreads();
    };

    Place kept = {0, 0};                          // all tokens
    u64 unused;
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const float top_p = a.top_p ? a.top_p[row] : 1.f;
    if (top_k > 0 && top_k < a.V) {
        // (tokens at -infinity are not counted: fewer may remain than top_k)
        u64 n = 0;
        for (int i = tid; i < a.V; i += ROW_THREADS) n += key_of(l[i]) != 0;
        n = wave_scan(n, lane);
        __syncthreads();
        if (lane == 63) waves[wave] = n;
        __syncthreads();
        n = 0;
        for (int w = 0; w < ROW_WAVES; ++w) n += waves[w];
        if ((u64)top_k < n) cut(Place{0, 0}, false, (u64)top_k, &kept, &unused);
    }

    // Sums over the chunks of what a place keeps; returns the whole sum.
    double min_weight = a.min_p ? (double)a.min_p[row] * ONE : 0.0;
    min_weight = min_weight > 0.0 ? min_weight : 0.0;
    auto keep = [&](u32 key, u64 w) { return key == top || (double)w >= min_weight; };
    const int chunks = (a.V + CHUNK - 1) / CHUNK;
    auto sums = [&](const Place &p, bool filter) {
        __syncthreads();
        for (int c = tid; c < chunks; c += ROW_THREADS) {
            chunk_weight[c] = 0;
            chunk_ties[c] = 0;
        }
        __syncthreads();
        for (int i = tid; i < a.V; i += ROW_THREADS) {
            const u32 key = key_of(l[i]);
            if (key > p.key) {
                const u64 w = weigh(key);
                if (w && (!filter || keep(key, w))) atomicAdd((unsigned long long *)&chunk_weight[i / CHUNK], w);
            } else if (key == p.key) {
                atomicAdd(&chunk_ties[i / CHUNK], 1u);
            }
        }
        __syncthreads();
    };
    u64 total = 0;
    if (top_p < 1.f) {
        sums(kept, false);
        for (int c = 0; c < chunks; ++c) total += chunk_weight[c];
        total += kept.ties * weigh(kept.key);
        const double want = ceil((double)top_p * (double)total);
        cut(kept, true, want >= 1.0 ? (want < (double)total ? (u64)want : total) : 1, &kept, &unused);
    }
    sums(kept, true);
    // the chunk and the token in it
    const u64 tie = kept.key && kept.ties ? weigh(kept.key) : 0;
    const u64 tie_kept = kept.key && keep(kept.key, tie) ? tie : 0;
    if (tid == 0) {
        u64 all = 0, ties = 0;
        for (int c = 0; c < chunks; ++c) {
            const u64 n = ties < kept.ties ? min((u64)chunk_ties[c], kept.ties - ties) : 0;
            ties += chunk_ties[c];
            chunk_weight[c] += n * tie_kept;
            all += chunk_weight[c];
        }
        const double u = a.u[row] > 0.f ? (double)a.u[row] : 0.0;
        const double at = u * (double)all;
        const u64 thr = at < (double)all ? min((u64)at, all - 1) : all - 1;
        u64 sum = 0, before = 0;
        int c = 0;
        for (; c < chunks - 1 && sum + chunk_weight[c] <= thr; ++c) {
            sum += chunk_weight[c];
            before += chunk_ties[c];
        }
        found[0] = (u64)c;
        found[1] = thr - sum;
        found[2] = before;
        waves[0] = all;
    }
    __syncthreads();
    const int c0 = (int)found[0] * CHUNK;
    const u64 thr = found[1], ties_before = found[2], all = waves[0];
    __syncthreads();
    // 4 tokens a thread, in order
    u32 key[4];
    u64 w[4], n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = c0 + 4 * tid + j;
        key[j] = i < a.V ? key_of(l[i]) : 0;
        n += key[j] && key[j] == kept.key;
    }
    u64 s = wave_scan(n, lane);
    if (lane == 63) waves[wave] = s;
    __syncthreads();
    u64 ties = ties_before + s - n;
    for (int v = 0; v < wave; ++v) ties += waves[v];
    __syncthreads();
    n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = 0;
        if (key[j] > kept.key) {
            w[j] = weigh(key[j]);
            if (!keep(key[j], w[j])) w[j] = 0;
        } else if (key[j] && key[j] == kept.key) {
            if (ties++ < kept.ties) w[j] = tie_kept;
        }
        n += w[j];
    }
    s = wave_scan(n, lane);
    if (lane == 63) waves[wave] = s;
    __syncthreads();
    u64 sum = s - n;
    for (int v = 0; v < wave; ++v) sum += waves[v];
    if (sum <= thr && sum + n > thr) {
        int j = 0;
        for (; j < 3 && sum + w[j] <= thr; ++j) sum += w[j];
        a.tokens[row] = c0 + 4 * tid + j;
        if (a.probs) a.probs[row] = (float)((double)w[j] / (double)all);
    }
}

} // namespace step
} // namespace kq

using namespace kq;
using namespace kq::step;

extern "C" {

size_t kqstep_sample_workspace_bytes(int M, int64_t V) {
    if (M < 0 || M > 65536 || V < 1 || V > MAX_V) return 0;
    return 16;
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
    if (workspace_bytes < kqstep_sample_workspace_bytes(M, V)) return KQ_ERR_SHAPE;
    if (device_check()) return KQ_ERR_DEVICE;
    const Sample a = {logits, temperature, top_p, min_p, u, top_k, tokens, probs, ld, (int)V};
    hipLaunchKernelGGL(sample_kernel, dim3((unsigned)M), dim3(ROW_THREADS), 0, (hipStream_t)stream, a);
    return kv::launched();
}

} // extern "C"
