// kq_kv.hip -- the page plan, the rotary positions with the cache store and
// the cache load of include/kqkv.h.
#include "kq_kv.h"

#include <cmath>

namespace kq {
namespace kv {

// ---------------------------------------------------------------------------
// Plan

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_WAVES = PLAN_THREADS / 64;
constexpr int SLOT_THREADS = 256;

struct Plan {
    const int32_t *ctx_len, *new_len, *held, *n_free;
    int32_t *table, *held_out, *free_pages, *n_free_out, *slots, *pos, *seq_start, *ctx_out, *err;
    int64_t stride;
    int B, P, T, n_pages;
};

// What one request does in this step.  `bad`: a value out of range.
struct Req {
    int64_t after;      // length with its new tokens
    int fresh;          // new tokens
    int need, gone;     // pages taken, pages given back
    int held;
    bool bad;
};

__device__ __forceinline__ Req plan_req(const Plan &p, int b) {
    Req r = {0, 0, 0, 0, 0, false};
    if (b >= p.B) return r;
    const int ctx = p.ctx_len[b], add = p.new_len[b], held = p.held[b];
    r.held = held;
    if (ctx < 0 || held < 0 || held > p.stride) {
        r.bad = true;
        return r;
    }
    if (add < 0) {
        r.gone = held;
        return r;
    }
    r.after = (int64_t)ctx + add;
    const int64_t pages = (r.after + p.P - 1) / p.P;
    if (pages > p.stride || r.after > INT32_MAX) {
        r.bad = true;
        return r;
    }
    r.fresh = add;
    r.need = pages > held ? (int)(pages - held) : 0;
    return r;
}

// Three running sums of a block: each thread's exclusive ones and the totals.
// Sums over all requests stay below 2^16 * 2^31.
struct Sums { int64_t fresh, need, gone; };
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}
__device__ __forceinline__ void block_scan(const Req &r, Sums *wave_sums, Sums *excl, Sums *total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Sums in = {wave_scan(r.fresh, lane), wave_scan(r.need, lane), wave_scan(r.gone, lane)};
    __syncthreads();                              // the last use of wave_sums is over
    if (lane == 63) wave_sums[wave] = in;
    __syncthreads();
    Sums e = {in.fresh - r.fresh, in.need - r.need, in.gone - r.gone}, t = {0, 0, 0};
    for (int w = 0; w < PLAN_WAVES; ++w) {
        const Sums s = wave_sums[w];
        if (w < wave) {
            e.fresh += s.fresh;
            e.need += s.need;
            e.gone += s.gone;
        }
        t.fresh += s.fresh;
        t.need += s.need;
        t.gone += s.gone;
    }
    *excl = e;
    *total = t;
}

// Last index b in [0, n) with first[b] <= i (first ascending, first[0] <= i).
template <class T> __device__ __forceinline__ int last_not_after(const T *first, int n, T i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// Slot and position of row t, from the outputs of the requests' part.
__device__ __forceinline__ void plan_row(const Plan &p, const int32_t *start, int t) {
    int pos = 0, slot = -1;
    if (t < start[p.B]) {
        const int b = last_not_after(start, p.B, t);
        pos = p.ctx_out[b] - (start[b + 1] - t);
        const u32 page = (u32)pos / (u32)p.P;
        const u32 id = (u32)p.table[(int64_t)b * p.stride + page];
        if (id < (u32)p.n_pages) slot = (int)(id * p.P + ((u32)pos - page * (u32)p.P));
    }
    p.pos[t] = pos;
    p.slots[t] = slot;
}

// One work-group for the requests: prefix sums of the new tokens and of the
// pages taken and given back, then the pages themselves, a thread per page (the
// request of page i by bisection of the prefix sums in LDS).  `rows`: it fills
// slots and pos too.
__global__ __launch_bounds__(PLAN_THREADS) void plan_kernel(Plan p, int rows) {
    __shared__ Sums wave_sums[PLAN_WAVES];
    __shared__ int first_need[PLAN_THREADS], first_gone[PLAN_THREADS], base[PLAN_THREADS];
    __shared__ int any_bad;
    const int tid = threadIdx.x;
    if (tid == 0) any_bad = 0;
    __syncthreads();
    // totals, before anything is written
    Sums total = {0, 0, 0}, excl;
    Req r;
    for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
        Sums t;
        r = plan_req(p, b0 + tid);
        if (r.bad) any_bad = 1;
        block_scan(r, wave_sums, &excl, &t);
        total.fresh += t.fresh;
        total.need += t.need;
        total.gone += t.gone;
    }
    const int64_t n_free = p.n_free[0];
    const int64_t top = n_free + total.gone;
    __syncthreads();
    const bool ok = !any_bad && n_free >= 0 && top <= p.n_pages && total.need <= top && total.fresh <= p.T;
    const bool one = p.B <= PLAN_THREADS;          // r and excl are still those of every request
    if (!ok) {
        for (int b = tid; b < p.B; b += PLAN_THREADS) {
            p.seq_start[b] = 0;
            p.held_out[b] = p.held[b];
            p.ctx_out[b] = p.ctx_len[b];
        }
        if (tid == 0) {
            p.seq_start[p.B] = 0;
            p.n_free_out[0] = (int)n_free;
            if (p.err) p.err[0] = 1;
        }
    } else {
        // the ended requests' pages go on the list first: in another order
        // than the requests' own chunks, so in a pass of their own
        Sums done = {0, 0, 0};
        for (int b0 = 0; total.gone > 0 && b0 < p.B; b0 += PLAN_THREADS) {
            Sums t;
            if (!one) {
                r = plan_req(p, b0 + tid);
                block_scan(r, wave_sums, &excl, &t);
            } else {
                t = total;
            }
            first_gone[tid] = (int)excl.gone;
            __syncthreads();
            const int n = p.B - b0 < PLAN_THREADS ? p.B - b0 : PLAN_THREADS;
            for (int i = tid; i < (int)t.gone; i += PLAN_THREADS) {
                const int b = last_not_after(first_gone, n, i);
                p.free_pages[n_free + done.gone + i] = p.table[(int64_t)(b0 + b) * p.stride + (i - first_gone[b])];
            }
            done.gone += t.gone;
            __syncthreads();
        }
        for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
            Sums t;
            const int b = b0 + tid;
            if (!one) {
                r = plan_req(p, b);
                block_scan(r, wave_sums, &excl, &t);
            } else {
                t = total;
            }
            first_need[tid] = (int)excl.need;
            base[tid] = r.held;
            __syncthreads();
            const int n = p.B - b0 < PLAN_THREADS ? p.B - b0 : PLAN_THREADS;
            for (int i = tid; i < (int)t.need; i += PLAN_THREADS) {
                const int c = last_not_after(first_need, n, i);
                p.table[(int64_t)(b0 + c) * p.stride + base[c] + (i - first_need[c])] =
                    p.free_pages[top - 1 - (done.need + i)];
            }
            if (b < p.B) {
                p.seq_start[b] = (int)(done.fresh + excl.fresh);
                p.held_out[b] = r.gone ? 0 : r.held + r.need;
                p.ctx_out[b] = (int)r.after;
            }
            done.fresh += t.fresh;
            done.need += t.need;
            __syncthreads();
        }
        if (tid == 0) {
            p.seq_start[p.B] = (int)total.fresh;
            p.n_free_out[0] = (int)(top - total.need);
        }
    }
    if (rows) {
        __threadfence_block();
        __syncthreads();
        for (int t = tid; t < p.T; t += PLAN_THREADS) plan_row(p, p.seq_start, t);
    }
}

__global__ __launch_bounds__(SLOT_THREADS) void plan_rows_kernel(Plan p) {
    const int t = blockIdx.x * SLOT_THREADS + threadIdx.x;
    if (t < p.T) plan_row(p, p.seq_start, t);
}

// ---------------------------------------------------------------------------
// Rotary positions and store

constexpr int STORE_THREADS = 256;
constexpr int MAX_DIM = 256, MAX_PAIRS = MAX_DIM / 2;

struct Rope {
    double log2_base;
    const float *factors;
    const int32_t *pos;
    int64_t pos_stride;
    int style, pairs;      // pairs 0: nothing turns
    int end[4];            // pair i takes the first axis a with i < end[a]
};

struct Rows {
    const float *q, *k, *v;
    float *q_out;
    int64_t ldq, ldq_out, ldk, ldv;
    int q_heads, T;
};

// Cosine and sine of pair i of token t.  The angle is taken in turns,
// t / 2 pi, so that its whole part drops out exactly.
__device__ __forceinline__ double2 rope_turn(const Rope &r, int t, int i) {
    const int axis = (i >= r.end[0]) + (i >= r.end[1]) + (i >= r.end[2]);
    double f = exp2(-2.0 * i / (2.0 * r.pairs) * r.log2_base);
    if (r.factors) f /= (double)r.factors[i];
    double turns = (double)r.pos[axis * r.pos_stride + t] * f * 0.15915494309189533577;
    turns -= rint(turns);
    double2 cs;
    sincospi(2.0 * turns, &cs.y, &cs.x);
    return cs;
}

__device__ __forceinline__ void rope_pair(const Rope &r, int i, int *a, int *b) {
    *a = r.style == KQKV_ROPE_HALVES ? i : 2 * i;
    *b = r.style == KQKV_ROPE_HALVES ? i + r.pairs : 2 * i + 1;
}

// Orders a wave's LDS writes before its other lanes' reads.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// One head's row of one token (in LDS, the wave's own) into the cache.
template <bool Q8, bool V>
__device__ __forceinline__ void store_row(const Cache &c, const float *row, u32 slot, int head, int lane) {
    const u32 page = slot / c.page_tokens, t = slot - page * c.page_tokens;
    uint8_t *to = (V ? c.v : c.k) + page * c.page_bytes + (u64)head * c.head_bytes;
    if (!Q8) {
        for (int d = lane; d < c.dim; d += 64)
            ((_Float16 *)to)[V ? v_at(t, d, c.dim) : k_at(t, d, c.dim)] = (_Float16)row[d];
        return;
    }
    _Float16 *scales = (_Float16 *)(to + c.page_tokens * c.dim);
    for (int d0 = 0; d0 < c.dim; d0 += 64) {           // a block of 32 in each half of the wave
        const int d = d0 + lane;
        const float x = d < c.dim ? row[d] : 0.f;
        u32 m = __builtin_bit_cast(u32, x) & 0x7FFFFFFFu;   // magnitudes order like integers, NaN on top
#pragma unroll
        for (int s = 16; s; s >>= 1) m = max(m, (u32)__shfl_xor((int)m, s));
        const bool bad = m >= 0x7F800000u;
        float s = (float)(_Float16)fminf(__builtin_bit_cast(float, m) / 127.f, 65504.f);
        const float n = s > 0.f && !bad ? rintf(x / s) : 0.f;
        if (bad) s = __builtin_nanf("");
        if (d < c.dim) {
            to[V ? v_at(t, d, c.dim) : k_at(t, d, c.dim)] = (uint8_t)(int8_t)fmaxf(-127.f, fminf(127.f, n));
            if ((lane & 31) == 0) scales[scale_at(t, d >> 5, c.dim)] = (_Float16)s;
        }
    }
}

template <bool Q8>
__global__ __launch_bounds__(STORE_THREADS) void rope_store_kernel(Cache c, Rope r, Rows x, const int32_t *slots) {
    __shared__ double2 cs[MAX_PAIRS];
    __shared__ float rows[STORE_THREADS / 64][MAX_DIM];
    const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < r.pairs; i += STORE_THREADS) cs[i] = rope_turn(r, t, i);
    __syncthreads();
    const u32 slot = x.k ? (u32)slots[t] : ~0u;
    const int heads = x.q_heads + (slot < c.slots ? 2 * c.kv_heads : 0);
    float *row = rows[wave];
    for (int h = wave; h < heads; h += STORE_THREADS / 64) {
        const int kh = h - x.q_heads, vh = kh - c.kv_heads;
        const float *in = kh < 0 ? x.q + t * x.ldq + (int64_t)h * c.dim
                        : vh < 0 ? x.k + t * x.ldk + (int64_t)kh * c.dim : x.v + t * x.ldv + (int64_t)vh * c.dim;
        const int pairs = vh < 0 ? r.pairs : 0;
        for (int i = lane; i < pairs; i += 64) {
            int a, b;
            rope_pair(r, i, &a, &b);
            const double va = in[a], vb = in[b];
            row[a] = (float)(va * cs[i].x - vb * cs[i].y);
            row[b] = (float)(va * cs[i].y + vb * cs[i].x);
        }
        for (int d = 2 * pairs + lane; d < c.dim; d += 64) row[d] = in[d];
        wave_sync();
        if (kh < 0) {
            for (int d = lane; d < c.dim; d += 64) x.q_out[t * x.ldq_out + (int64_t)h * c.dim + d] = row[d];
        } else if (vh < 0) {
            store_row<Q8, false>(c, row, slot, kh, lane);
        } else {
            store_row<Q8, true>(c, row, slot, vh, lane);
        }
        wave_sync();
    }
}

// ---------------------------------------------------------------------------
// Load

template <bool Q8, bool V>
__device__ __forceinline__ float cached(const Cache &c, u32 page, u32 t, int head, int d) {
    const uint8_t *from = (V ? c.v : c.k) + page * c.page_bytes + (u64)head * c.head_bytes;
    const u32 i = V ? v_at(t, d, c.dim) : k_at(t, d, c.dim);
    if (!Q8) return (float)((const _Float16 *)from)[i];
    return (float)((const _Float16 *)(from + c.page_tokens * c.dim))[scale_at(t, d >> 5, c.dim)] *
           (float)((const int8_t *)from)[i];
}

template <bool Q8>
__global__ __launch_bounds__(STORE_THREADS) void load_kernel(Cache c, const int32_t *slots, float *k, float *v) {
    const int t = blockIdx.x, n = c.kv_heads * c.dim;
    const u32 slot = (u32)slots[t];
    if (slot >= c.slots) return;
    const u32 page = slot / c.page_tokens, at = slot - page * c.page_tokens;
    for (int i = threadIdx.x; i < n; i += STORE_THREADS) {
        const int head = i / c.dim, d = i - head * c.dim;
        if (k) k[(int64_t)t * n + i] = cached<Q8, false>(c, page, at, head, d);
        if (v) v[(int64_t)t * n + i] = cached<Q8, true>(c, page, at, head, d);
    }
}

} // namespace kv
} // namespace kq

using namespace kq;
using namespace kq::kv;

extern "C" {

int64_t kqkv_page_bytes(int type, int kv_heads, int head_dim, int page_tokens) {
    const int r = cache_limits(type, kv_heads, head_dim, page_tokens);
    if (r) return r;
    const int64_t n = (int64_t)kv_heads * head_dim * page_tokens;
    return type == KQKV_F16 ? 2 * n : n + n / 16;
}

int kqkv_plan(int B, const int32_t *ctx_len, const int32_t *new_len, int page_tokens, int32_t *table,
              int64_t table_stride, const int32_t *held, int32_t *held_out, int32_t *free_pages, int64_t n_pages,
              const int32_t *n_free, int32_t *n_free_out, int T, int32_t *slots, int32_t *pos, int32_t *seq_start,
              int32_t *ctx_out, int32_t *err_flag, void *stream) {
    if (B < 1 || B > 65536 || T < 0 || table_stride < 1 || table_stride > (1 << 24)) return KQ_ERR_SHAPE;
    if (page_tokens < 16 || page_tokens > 256 || page_tokens % 16) return KQ_ERR_SHAPE;
    if (n_pages < 1 || n_pages > INT32_MAX / page_tokens) return KQ_ERR_SHAPE;
    const void *need[] = {ctx_len, new_len, table, held, held_out, free_pages, n_free, n_free_out, seq_start, ctx_out};
    for (const void *a : need)
        if (!a) return KQ_ERR_NULL;
    if (T && (!slots || !pos)) return KQ_ERR_NULL;
    for (const void *a : need)
        if (!aligned(a, 4)) return KQ_ERR_ALIGN;
    if (!aligned(slots, 4) || !aligned(pos, 4) || !aligned(err_flag, 4)) return KQ_ERR_ALIGN;
    if (device_check()) return KQ_ERR_DEVICE;
    Plan p = {ctx_len, new_len, held, n_free, table, held_out, free_pages, n_free_out, slots, pos, seq_start, ctx_out,
              err_flag, table_stride, B, page_tokens, T, (int)n_pages};
    hipStream_t st = (hipStream_t)stream;
    const bool apart = T > 4 * PLAN_THREADS;
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, st, p, apart ? 0 : 1);
    if (apart)
        hipLaunchKernelGGL(plan_rows_kernel, dim3((unsigned)(((int64_t)T + SLOT_THREADS - 1) / SLOT_THREADS)),
                           dim3(SLOT_THREADS), 0, st, p);
    return launched();
}

int kqkv_rope_store(const kqkv_cache *cache, const kqkv_rope *rope, int T, const int32_t *pos, int64_t pos_stride,
                    const int32_t *slots, int q_heads, const float *q, int64_t ldq, float *q_out, int64_t ldq_out,
                    const float *k, int64_t ldk, const float *v, int64_t ldv, void *stream) {
    int r = cache_check(cache);
    if (r) return r;
    if (T < 0 || T >= (1 << 24) || q_heads < 0 || q_heads > 1024) return KQ_ERR_SHAPE;
    Rope ra = {};
    if (rope) {
        if (rope->style != KQKV_ROPE_HALVES && rope->style != KQKV_ROPE_PAIRS) return KQ_ERR_ARG;
        if (rope->rot_dims < 2 || rope->rot_dims % 2 || rope->rot_dims > cache->head_dim) return KQ_ERR_SHAPE;
        if (!(rope->base > 0.f) || !std::isfinite(rope->base)) return KQ_ERR_ARG;
        if (rope->n_axes < 1 || rope->n_axes > 4) return KQ_ERR_ARG;
        ra.pairs = rope->rot_dims / 2;
        int64_t sum = 0;
        for (int a = 0; a < 4; ++a) {
            if (a < rope->n_axes) {
                if (rope->sections[a] < 0) return KQ_ERR_ARG;
                sum += rope->sections[a];
            }
            ra.end[a] = (int)std::min<int64_t>(sum, ra.pairs);
        }
        if (sum != ra.pairs) return KQ_ERR_ARG;
        if (T > 0 && rope->n_axes > 1 && pos_stride < T) return KQ_ERR_SHAPE;
    } else if (q_heads) {
        return KQ_ERR_ARG;
    }
    if ((k == nullptr) != (v == nullptr)) return KQ_ERR_NULL;
    if (T == 0 || (!q_heads && !k)) return KQ_OK;
    if (rope && !pos) return KQ_ERR_NULL;
    if (k && !slots) return KQ_ERR_NULL;
    if (!aligned(pos, 4) || !aligned(slots, 4) || (rope && !aligned(rope->freq_factors, 4))) return KQ_ERR_ALIGN;
    const int64_t nq = (int64_t)q_heads * cache->head_dim, nk = (int64_t)cache->kv_heads * cache->head_dim;
    if (q_heads && ((r = rows_check(q, ldq, nq)) || (r = rows_check(q_out, ldq_out, nq)))) return r;
    if (k && ((r = rows_check(k, ldk, nk)) || (r = rows_check(v, ldv, nk)))) return r;
    if (q_heads && q == q_out && ldq != ldq_out) return KQ_ERR_ARG;
    if (device_check()) return KQ_ERR_DEVICE;
    if (rope) {
        ra.log2_base = std::log2((double)rope->base);
        ra.factors = rope->freq_factors;
        ra.pos = pos;
        ra.pos_stride = pos_stride;
        ra.style = rope->style;
    }
    const Rows x = {q, k, v, q_out, ldq, ldq_out, ldk, ldv, q_heads, T};
    hipStream_t st = (hipStream_t)stream;
    if (cache->type == KQKV_F16)
        hipLaunchKernelGGL(rope_store_kernel<false>, dim3(T), dim3(STORE_THREADS), 0, st, cache_args(cache), ra, x, slots);
    else
        hipLaunchKernelGGL(rope_store_kernel<true>, dim3(T), dim3(STORE_THREADS), 0, st, cache_args(cache), ra, x, slots);
    return launched();
}

int kqkv_load(const kqkv_cache *cache, int T, const int32_t *slots, float *k, float *v, void *stream) {
    const int r = cache_check(cache);
    if (r) return r;
    if (T < 0 || T >= (1 << 24)) return KQ_ERR_SHAPE;
    if (T == 0 || (!k && !v)) return KQ_OK;
    if (!slots) return KQ_ERR_NULL;
    if (!aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16)) return KQ_ERR_ALIGN;
    if (device_check()) return KQ_ERR_DEVICE;
    hipStream_t st = (hipStream_t)stream;
    if (cache->type == KQKV_F16)
        hipLaunchKernelGGL(load_kernel<false>, dim3(T), dim3(STORE_THREADS), 0, st, cache_args(cache), slots, k, v);
    else
        hipLaunchKernelGGL(load_kernel<true>, dim3(T), dim3(STORE_THREADS), 0, st, cache_args(cache), slots, k, v);
    return launched();
}

} // extern "C"
