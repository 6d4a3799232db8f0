// kq_kv.hip -- the page plan, the rotary positions with the cache store and
// the cache load of include/kqkv.h.
#include "kq_kv.h"

#include <cmath>

namespace kq {
namespace kv {

// ---------------------------------------------------------------------------
// Plan
//
// Bound: latency.  One work-group holds up to 1024 requests (256 where that
// suffices, and few rows: its barriers are shorter, 16 requests and rows 5.2 ->
// 4.4 us, but 3600 pages for 256 requests 6.9 -> 14.9), one a thread:
// prefix sums of the new tokens and of the pages taken and given back, then a
// thread per page and per row, which find their request by bisection in LDS.
// Few rows are filled in by the same work-group, from the free list and the
// table as they were, beside the writes; many by a second launch.

constexpr int PLAN_THREADS = 1024, PLAN_FEW = 256;
constexpr int ROW_THREADS = 256, ROW_STARTS = 4096;

struct Plan {
    const int32_t *ctx_len, *new_len, *held, *n_free;
    int32_t *table, *held_out, *free_pages, *n_free_out, *slots, *pos, *seq_start, *ctx_out, *err;
    int64_t stride;
    int B, P, T, n_pages;
};

// What one request does in this step.  `bad`: a value out of range.
struct Req {
    int after;          // length with its new tokens
    int fresh;          // new tokens, at most T < 2^23
    int need, gone;     // pages taken, pages given back, at most 2^24
    int held;
    bool bad;
};

__device__ __forceinline__ Req plan_req(const Plan &p, int b) {
    const bool in = b < p.B;
    const int i = in ? b : 0;
    const int ctx = p.ctx_len[i], add = p.new_len[i], held = p.held[i];
    Req r = {0, 0, 0, 0, held, false};
    if (!in) return r;
    if (ctx < 0 || held < 0 || held > p.stride) {
        r.bad = true;
    } else if (add < 0) {
        r.gone = held;
    } else {
        const int64_t after = (int64_t)ctx + add;
        const u32 pages = after > INT32_MAX ? ~0u : ((u32)after + (u32)p.P - 1) / (u32)p.P;
        if (pages > p.stride || add > p.T) {
            r.bad = true;
        } else {
            r.after = (int)after;
            r.fresh = add;
            r.need = max((int)pages - held, 0);
        }
    }
    return r;
}

// Inclusive prefix sums over a wave (or, ROWS_ONLY, over each row of 16 lanes).
template <int CTRL, int ROWS> __device__ __forceinline__ int dpp_or_0(int x) {
    return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
template <bool ROWS_ONLY> __device__ __forceinline__ int scan(int x) {
    x += dpp_or_0<0x111, 0xF>(x);
    x += dpp_or_0<0x112, 0xF>(x);
    x += dpp_or_0<0x114, 0xF>(x);
    x += dpp_or_0<0x118, 0xF>(x);
    if (!ROWS_ONLY) {
        x += dpp_or_0<0x142, 0xA>(x);
        x += dpp_or_0<0x143, 0xC>(x);
    }
    return x;
}

// A running sum over the work-group's threads: each thread's exclusive one and
// the total.  A wave's sum stays below 2^30, the total is held in 64 bits (where
// it passes 31, the step fails and the exclusive sums are not used).
struct Sum { int before; int64_t total; };
template <int WAVES> __device__ __forceinline__ Sum block_sum(int x, int scanned, const int *waves, int wave) {
    const int lane = threadIdx.x & 63, w = (lane & 15) < WAVES ? waves[lane & (WAVES - 1)] : 0;
    const int s = scan<true>(w);
    const int64_t total = ((int64_t)__builtin_amdgcn_readlane(scan<true>(w >> 16), 15) << 16) +
                          __builtin_amdgcn_readlane(scan<true>(w & 0xFFFF), 15);
    return Sum{__builtin_amdgcn_readlane(s - w, wave) + scanned - x, total};
}
struct Sums { Sum fresh, need, gone; };
template <int WAVES> __device__ __forceinline__ Sums block_sums(const Req &r, int (*waves)[WAVES]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int f = scan<false>(r.fresh), n = scan<false>(r.need), g = scan<false>(r.gone);
    __syncthreads();                              // the last use of `waves` is over
    if (lane == 63) {
        waves[0][wave] = f;
        waves[1][wave] = n;
        waves[2][wave] = g;
    }
    __syncthreads();
    return Sums{block_sum<WAVES>(r.fresh, f, waves[0], wave), block_sum<WAVES>(r.need, n, waves[1], wave),
                block_sum<WAVES>(r.gone, g, waves[2], wave)};
}

// Last index b in [0, n) with first[b] <= i (first ascending, first[0] <= i).
__device__ __forceinline__ int last_not_after(const int *first, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int slot_of(const Plan &p, u32 id, u32 pos, u32 page) {
    return id < (u32)p.n_pages ? (int)(id * p.P + (pos - page * (u32)p.P)) : -1;
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void plan_kernel(Plan p, int rows) {
    __shared__ int waves[3][THREADS / 64];
    __shared__ int first[THREADS], first_need[THREADS], after[THREADS], had[THREADS];
    const int tid = threadIdx.x;
    const bool one = p.B <= THREADS;
    const int n_free = p.n_free[0];
    // totals, before anything is written
    Req r = plan_req(p, tid);
    bool bad = r.bad;
    Sums s = block_sums(r, waves);
    int64_t fresh = s.fresh.total, need = s.need.total, gone = s.gone.total;
    for (int b0 = THREADS; b0 < p.B; b0 += THREADS) {
        const Req o = plan_req(p, b0 + tid);
        bad = bad || o.bad;
        const Sums t = block_sums(o, waves);
        fresh += t.fresh.total;
        need += t.need.total;
        gone += t.gone.total;
    }
    const int64_t top = n_free + gone;
    const bool ok = !__syncthreads_or(bad) && n_free >= 0 && top <= p.n_pages && need <= top && fresh <= p.T;
    if (!ok) {
        for (int b = tid; b < p.B; b += THREADS) {
            p.seq_start[b] = 0;
            p.held_out[b] = p.held[b];
            p.ctx_out[b] = p.ctx_len[b];
        }
        if (tid == 0) {
            p.seq_start[p.B] = 0;
            p.n_free_out[0] = n_free;
            if (p.err) p.err[0] = 1;
        }
        for (int t = tid; rows && t < p.T; t += THREADS) {
            p.slots[t] = -1;
            p.pos[t] = 0;
        }
        return;
    }
    // the ended requests' pages go on the list before any are taken from it
    if (gone) {
        int64_t done = n_free;
        for (int b0 = 0; b0 < p.B; b0 += THREADS) {
            if (!one) {
                r = plan_req(p, b0 + tid);
                s = block_sums(r, waves);
            }
            first[tid] = s.gone.before;
            __syncthreads();
            const int n = min(p.B - b0, THREADS);
            for (int i = tid; i < (int)s.gone.total; i += THREADS) {
                const int b = last_not_after(first, n, i);
                p.free_pages[done + i] = p.table[(int64_t)(b0 + b) * p.stride + (i - first[b])];
            }
            done += s.gone.total;
            __syncthreads();
        }
        __threadfence_block();
    }
    int tokens = 0, taken = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        if (!one) {
            r = plan_req(p, b0 + tid);
            s = block_sums(r, waves);
        }
        first[tid] = s.fresh.before;
        first_need[tid] = s.need.before;
        after[tid] = r.after;
        had[tid] = r.held;
        __syncthreads();
        const int n = min(p.B - b0, THREADS), b = b0 + tid;
        auto new_page = [&](int i) { return p.free_pages[top - 1 - (taken + i)]; };
        // rows (only where one chunk holds every request): their pages from the list and the table as they were
        for (int t = tid; rows && t < p.T; t += THREADS) {
            int pos = 0, slot = -1;
            if (t < (int)fresh) {
                const int c = last_not_after(first, n, t);
                const int end = c + 1 < n ? first[c + 1] : (int)fresh;
                pos = after[c] - (end - t);
                const u32 page = (u32)pos / (u32)p.P;
                const int at = (int)page - had[c];
                slot = slot_of(p, (u32)(at < 0 ? p.table[(int64_t)c * p.stride + page] : new_page(first_need[c] + at)), (u32)pos, page);
            }
            p.pos[t] = pos;
            p.slots[t] = slot;
        }
        for (int i = tid; i < (int)s.need.total; i += THREADS) {
            const int c = last_not_after(first_need, n, i);
            p.table[(int64_t)(b0 + c) * p.stride + had[c] + (i - first_need[c])] = new_page(i);
        }
        if (b < p.B) {
            p.seq_start[b] = tokens + s.fresh.before;
            p.held_out[b] = r.gone ? 0 : r.held + r.need;
            p.ctx_out[b] = r.after;
        }
        tokens += (int)s.fresh.total;
        taken += (int)s.need.total;
        __syncthreads();
    }
    if (tid == 0) {
        p.seq_start[p.B] = tokens;
        p.n_free_out[0] = (int)top - taken;
    }
}

// Rows, from the outputs of plan_kernel.
__global__ __launch_bounds__(ROW_THREADS) void plan_rows_kernel(Plan p) {
    __shared__ int starts[ROW_STARTS];
    const int t = blockIdx.x * ROW_THREADS + threadIdx.x;
    const bool here = p.B <= ROW_STARTS;
    if (here) {
        for (int b = threadIdx.x; b < p.B; b += ROW_THREADS) starts[b] = p.seq_start[b];
        __syncthreads();
    }
    if (t >= p.T) return;
    int pos = 0, slot = -1;
    if (t < p.seq_start[p.B]) {
        const int b = here ? last_not_after(starts, p.B, t) : last_not_after(p.seq_start, p.B, t);
        pos = p.ctx_out[b] - (p.seq_start[b + 1] - t);
        const u32 page = (u32)pos / (u32)p.P;
        slot = slot_of(p, (u32)p.table[(int64_t)b * p.stride + page], (u32)pos, page);
    }
    p.pos[t] = pos;
    p.slots[t] = slot;
}

// ---------------------------------------------------------------------------
// Rotary positions and store
//
// Bound: HBM (q is read and written, k and v read, once).  A lane takes 8
// elements of a head's row, 4 pairs or 8 that do not turn, as two 16-byte loads
// and stores, so dim / 8 lanes make a row and a wave takes 64 / (dim / 8) rows at
// a time; a work-group is one token and its waves go through the token's q and k
// rows, so that the token's angles (64-bit exponentials, sines and cosines) are
// computed once, while the first rows are on their way.  For few tokens the rows
// are spread over more work-groups.  v goes into the transposed groups of 16
// tokens: a wave takes 16 tokens by 32 elements, lane (t, i) elements 4 i .. of
// token t: 128 bytes of a row a token, and stores in which 16 lanes write
// neighbours where the tokens have neighbouring slots (no staging in LDS).

constexpr int STORE_THREADS = 256, STORE_WAVES = STORE_THREADS / 64;
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
    const int32_t *slots;
    int64_t ldq, ldq_out, ldk, ldv;
    int q_heads, T;
    int split;             // work-groups a token's q and k rows are spread over
    int v_wgs;             // work-groups of v, the first ones of the grid
    u32 lanes_magic;       // ceil(2^16 / (dim / 8)): lane / (dim / 8) = lane * magic >> 16
};

// Cosine and sine of pair i of token t.  The angle is taken in turns,
// t / 2 pi, so that its whole part drops out exactly.
__device__ __forceinline__ double2 rope_turn(const Rope &r, int t, int i) {
    const int axis = (i >= r.end[0]) + (i >= r.end[1]) + (i >= r.end[2]);
    const double at = (double)r.pos[axis * r.pos_stride + t];
    double f = exp2(-2.0 * i / (2.0 * r.pairs) * r.log2_base);
    if (r.factors) f /= (double)r.factors[i];
    double turns = at * f * 0.15915494309189533577;
    turns -= rint(turns);
    double2 cs;
    sincospi(2.0 * turns, &cs.y, &cs.x);
    return cs;
}

// Orders a wave's LDS writes before its other lanes' reads.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 4 elements at d of one head's row of one token into K.
template <bool Q8>
__device__ __forceinline__ void store_k4(const Cache &c, uint8_t *head, u32 t, int d, f4 x, u32 block_max) {
    if (!Q8) {
        *(h4 *)(head + 2 * k_at(t, d, c.dim)) = __builtin_convertvector(x, h4);
        return;
    }
    const Scale s = block_scale(block_max);
    u32 w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= ((u32)quant(x[i], s) & 0xFFu) << (8 * i);
    *(u32 *)(head + k_at(t, d, c.dim)) = w;
    if ((d & 31) == 0) ((_Float16 *)(head + c.page_tokens * c.dim))[scale_at(t, d >> 5, c.dim)] = (_Float16)s.s;
}

// 16 tokens by 32 elements of v, for the unit-th (tokens, head, elements).
template <bool Q8> __device__ __forceinline__ void store_v(const Cache &c, const Rows &x, int64_t unit, int lane) {
    const int blocks = c.dim >> 5, per = c.kv_heads * blocks;
    const int tokens = (int)(unit / per), left = (int)(unit - (int64_t)tokens * per), head = left / blocks, b = left - head * blocks;
    const int t = tokens * 16 + (lane & 15), i = lane >> 4;
    const u32 slot = t < x.T ? (u32)x.slots[t] : ~0u;
    const bool in = slot < c.slots;
    const float *from = x.v + (in ? t : 0) * x.ldv + (int64_t)head * c.dim + b * 32 + 4 * i;
    const f4 y[2] = {*(const f4 *)from, *(const f4 *)(from + 16)};
    const u32 page = slot / c.page_tokens, at = slot - page * c.page_tokens;
    uint8_t *to = c.v + (in ? page : 0) * c.page_bytes + (u64)head * c.head_bytes;
    u32 m = max(magnitude(y[0]), magnitude(y[1]));
    if (Q8) {
        m = max(m, (u32)__shfl_xor((int)m, 16));
        m = max(m, (u32)__shfl_xor((int)m, 32));
    }
    if (!in) return;
    const Scale s = block_scale(m);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const u32 j = v_at(at, b * 32 + 16 * k + 4 * i + e, c.dim);
            if (Q8) to[j] = (uint8_t)quant(y[k][e], s);
            else ((_Float16 *)to)[j] = (_Float16)y[k][e];
        }
    if (Q8 && i == 0) ((_Float16 *)(to + c.page_tokens * c.dim))[scale_at(at, b, c.dim)] = (_Float16)s.s;
}

// Needs rot_dims a multiple of 8 (all 4 pairs of a lane turn, or none).
template <bool Q8>
__global__ __launch_bounds__(STORE_THREADS) void rope_store_kernel(Cache c, Rope r, Rows x) {
    __shared__ double2 cs[MAX_PAIRS];
    __shared__ u32 block_max[STORE_WAVES][16 * 8];       // [wave][row of the wave][block of 32]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((int)blockIdx.x < x.v_wgs) {
        const int64_t units = (int64_t)((x.T + 15) / 16) * c.kv_heads * (c.dim >> 5);
        for (int64_t u = (int64_t)blockIdx.x * STORE_WAVES + wave; u < units; u += (int64_t)x.v_wgs * STORE_WAVES)
            store_v<Q8>(c, x, u, lane);
        return;
    }
    const int wg = blockIdx.x - x.v_wgs, t = wg / x.split, part = wg - t * x.split;
    const int lanes = c.dim >> 3, sub = (int)(((u32)lane * x.lanes_magic) >> 16), j = lane - sub * lanes;
    const int rows_a_wave = (int)((64 * x.lanes_magic) >> 16);
    const int rows = x.q_heads + (x.k ? c.kv_heads : 0), step = rows_a_wave * STORE_WAVES * x.split;
    const bool turns = j < (r.pairs >> 2);
    const int oa = turns && r.style == KQKV_ROPE_HALVES ? 4 * j : 8 * j, ob = turns && r.style == KQKV_ROPE_HALVES ? r.pairs + 4 * j : 8 * j + 4;
    const float *qrow = x.q + t * x.ldq, *krow = x.k + t * x.ldk;
    auto row_at = [&](int h) { return h < x.q_heads ? qrow + (int64_t)h * c.dim : krow + (int64_t)(h - x.q_heads) * c.dim; };
    int h = (part * STORE_WAVES + wave) * rows_a_wave + sub;
    const bool lane_in = sub < rows_a_wave;
    // the first rows are asked for before the angles are computed
    f4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    if (lane_in && h < rows) {
        const float *p = row_at(h);
        a = *(const f4 *)(p + oa);
        b = *(const f4 *)(p + ob);
    }
    const u32 slot = x.k ? (u32)x.slots[t] : ~0u;
    for (int i = threadIdx.x; i < r.pairs; i += STORE_THREADS) cs[i] = rope_turn(r, t, i);
    __syncthreads();
    double2 turn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) turn[i] = turns ? cs[4 * j + i] : double2{1.0, 0.0};
    const bool stored = slot < c.slots;
    const u32 page = stored ? slot / c.page_tokens : 0, at = slot - page * c.page_tokens;
    uint8_t *kpage = c.k + page * c.page_bytes;
    u32 *maxes = block_max[wave] + sub * 8;
    for (int h0 = h - sub; h0 < rows; h0 += step, h += step) {
        // the next rows, while these are turned
        f4 na = {0.f, 0.f, 0.f, 0.f}, nb = na;
        if (lane_in && h + step < rows) {
            const float *p = row_at(h + step);
            na = *(const f4 *)(p + oa);
            nb = *(const f4 *)(p + ob);
        }
        const bool mine = lane_in && h < rows, is_k = h >= x.q_heads;
        f4 ya = a, yb = b;
        if (turns) {
            if (r.style == KQKV_ROPE_HALVES) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const double va = a[i], vb = b[i];
                    ya[i] = (float)(va * turn[i].x - vb * turn[i].y);
                    yb[i] = (float)(va * turn[i].y + vb * turn[i].x);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const double va = i < 2 ? a[2 * i] : b[2 * i - 4], vb = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
                    const float u = (float)(va * turn[i].x - vb * turn[i].y), w = (float)(va * turn[i].y + vb * turn[i].x);
                    if (i < 2) {
                        ya[2 * i] = u;
                        ya[2 * i + 1] = w;
                    } else {
                        yb[2 * i - 4] = u;
                        yb[2 * i - 3] = w;
                    }
                }
            }
        }
        if (mine && !is_k) {
            float *p = x.q_out + t * x.ldq_out + (int64_t)h * c.dim;
            *(f4 *)(p + oa) = ya;
            *(f4 *)(p + ob) = yb;
        }
        if (h0 + rows_a_wave > x.q_heads && stored) {        // some of the wave's rows are k's
            u32 ma = 0, mb = 0;
            if (Q8) {
                // the blocks' largest magnitudes: 4 elements lie in one block, a lane's two fours in any two
                for (int i = lane; i < 16 * 8; i += 64) block_max[wave][i] = 0;
                wave_sync();
                if (mine) {
                    atomicMax(&maxes[oa >> 5], magnitude(ya));
                    atomicMax(&maxes[ob >> 5], magnitude(yb));
                }
                wave_sync();
                if (mine) {
                    ma = maxes[oa >> 5];
                    mb = maxes[ob >> 5];
                }
                wave_sync();
            }
            if (mine && is_k) {
                uint8_t *head = kpage + (u64)(h - x.q_heads) * c.head_bytes;
                store_k4<Q8>(c, head, at, oa, ya, ma);
                store_k4<Q8>(c, head, at, ob, yb, mb);
            }
        }
        a = na;
        b = nb;
    }
}

// Any even rot_dims: a pair a lane, q and k only (k through LDS).  Loads and
// stores of 4 bytes a lane, one work-group a token: 64 query and 8 kv heads of 128,
// 126 of them turning, 9.5 us for one token and 88 for 4099 (fp16; Q8_0 12.5 and
// 105), where rot_dims of a multiple of 8 are at 2.9 us and the copy's rate.
template <bool Q8>
__global__ __launch_bounds__(STORE_THREADS) void rope_store_any_kernel(Cache c, Rope r, Rows x) {
    __shared__ double2 cs[MAX_PAIRS];
    __shared__ __align__(16) float rows[STORE_WAVES][MAX_DIM];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((int)blockIdx.x < x.v_wgs) {
        const int64_t units = (int64_t)((x.T + 15) / 16) * c.kv_heads * (c.dim >> 5);
        for (int64_t u = (int64_t)blockIdx.x * STORE_WAVES + wave; u < units; u += (int64_t)x.v_wgs * STORE_WAVES)
            store_v<Q8>(c, x, u, lane);
        return;
    }
    const int t = blockIdx.x - x.v_wgs;
    for (int i = threadIdx.x; i < r.pairs; i += STORE_THREADS) cs[i] = rope_turn(r, t, i);
    __syncthreads();
    const u32 slot = x.k ? (u32)x.slots[t] : ~0u;
    const int heads = x.q_heads + (slot < c.slots ? c.kv_heads : 0);
    const u32 page = slot / c.page_tokens, at = slot - page * c.page_tokens;
    float *row = rows[wave];
    for (int h = wave; h < heads; h += STORE_WAVES) {
        const int kh = h - x.q_heads;
        const float *in = kh < 0 ? x.q + t * x.ldq + (int64_t)h * c.dim : x.k + t * x.ldk + (int64_t)kh * c.dim;
        for (int i = lane; i < r.pairs; i += 64) {
            const int a = r.style == KQKV_ROPE_HALVES ? i : 2 * i, b = r.style == KQKV_ROPE_HALVES ? i + r.pairs : 2 * i + 1;
            const double va = in[a], vb = in[b];
            row[a] = (float)(va * cs[i].x - vb * cs[i].y);
            row[b] = (float)(va * cs[i].y + vb * cs[i].x);
        }
        for (int d = 2 * r.pairs + lane; d < c.dim; d += 64) row[d] = in[d];
        wave_sync();
        if (kh < 0) {
            for (int d = lane; d < c.dim; d += 64) x.q_out[t * x.ldq_out + (int64_t)h * c.dim + d] = row[d];
        } else {
            uint8_t *head = c.k + page * c.page_bytes + (u64)kh * c.head_bytes;
            for (int d = 4 * lane; d < c.dim; d += 256) {
                u32 m = 0;
                if (Q8)
                    for (int e = d & ~31; e < (d & ~31) + 32; e += 4) m = max(m, magnitude(*(const f4 *)(row + e)));
                store_k4<Q8>(c, head, at, d, *(const f4 *)(row + d), m);
            }
        }
        wave_sync();
    }
}

// ---------------------------------------------------------------------------
// Load: K by rows, 4 elements a lane, V in the units of the store.  HBM: 8192
// tokens of 8 heads of 128 23.5 us from fp16 (4.3 TB/s) and from Q8_0 23.4 (3.6).

template <bool Q8>
__device__ __forceinline__ void load_v4(const Cache &c, const int32_t *slots, int T, float *v, int64_t unit, int lane) {
    const int blocks = c.dim >> 5, per = c.kv_heads * blocks;
    const int tokens = (int)(unit / per), left = (int)(unit - (int64_t)tokens * per), head = left / blocks, b = left - head * blocks;
    const int t = tokens * 16 + (lane & 15), i = lane >> 4;
    const u32 slot = t < T ? (u32)slots[t] : ~0u;
    if (slot >= c.slots) return;
    const u32 page = slot / c.page_tokens, at = slot - page * c.page_tokens;
    const uint8_t *from = c.v + page * c.page_bytes + (u64)head * c.head_bytes;
    const float s = Q8 ? (float)((const _Float16 *)(from + c.page_tokens * c.dim))[scale_at(at, b, c.dim)] : 1.f;
    float *to = v + ((int64_t)t * c.kv_heads + head) * c.dim + b * 32 + 4 * i;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        f4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const u32 j = v_at(at, b * 32 + 16 * k + 4 * i + e, c.dim);
            y[e] = Q8 ? s * (float)((const int8_t *)from)[j] : (float)((const _Float16 *)from)[j];
        }
        *(f4 *)(to + 16 * k) = y;
    }
}

template <bool Q8>
__global__ __launch_bounds__(STORE_THREADS) void load_kernel(Cache c, const int32_t *slots, int T, float *k, float *v, int v_wgs) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((int)blockIdx.x < v_wgs) {
        const int64_t units = (int64_t)((T + 15) / 16) * c.kv_heads * (c.dim >> 5);
        for (int64_t u = (int64_t)blockIdx.x * STORE_WAVES + wave; u < units; u += (int64_t)v_wgs * STORE_WAVES)
            load_v4<Q8>(c, slots, T, v, u, lane);
        return;
    }
    const int t = blockIdx.x - v_wgs, n = c.kv_heads * c.dim;
    const u32 slot = (u32)slots[t];
    if (slot >= c.slots) return;
    const u32 page = slot / c.page_tokens, at = slot - page * c.page_tokens;
    for (int i = 4 * threadIdx.x; i < n; i += 4 * STORE_THREADS) {
        const int head = i / c.dim, d = i - head * c.dim;
        const uint8_t *from = c.k + page * c.page_bytes + (u64)head * c.head_bytes;
        f4 y;
        if (Q8) {
            const float s = (float)((const _Float16 *)(from + c.page_tokens * c.dim))[scale_at(at, d >> 5, c.dim)];
            const u32 w = *(const u32 *)(from + k_at(at, d, c.dim));
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = s * (float)(int8_t)(w >> (8 * e));
        } else {
            y = __builtin_convertvector(*(const h4 *)(from + 2 * k_at(at, d, c.dim)), f4);
        }
        *(f4 *)(k + (int64_t)t * n + i) = y;
    }
}

// Work-groups for the units of v (16 tokens, head, 32 elements), a wave each as
// long as the grid allows it.
static int v_workgroups(const kqkv_cache *c, int T) {
    const int64_t units = (int64_t)((T + 15) / 16) * c->kv_heads * (c->head_dim / 32);
    return (int)std::min<int64_t>((units + STORE_WAVES - 1) / STORE_WAVES, 1 << 22);
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
    if (B < 1 || B > 65536 || T < 0 || T >= (1 << 23) || table_stride < 1 || table_stride > (1 << 24)) return KQ_ERR_SHAPE;
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
    // a work-group alone fills in 4 rows a thread as fast as a second launch begins
    const bool apart = T > 4 * PLAN_THREADS || B > PLAN_THREADS;
    if (B <= PLAN_FEW && T <= 4 * PLAN_FEW)
        hipLaunchKernelGGL(plan_kernel<PLAN_FEW>, dim3(1), dim3(PLAN_FEW), 0, st, p, apart ? 0 : 1);
    else
        hipLaunchKernelGGL(plan_kernel<PLAN_THREADS>, dim3(1), dim3(PLAN_THREADS), 0, st, p, apart ? 0 : 1);
    if (apart && T)
        hipLaunchKernelGGL(plan_rows_kernel, dim3((unsigned)((T + ROW_THREADS - 1) / ROW_THREADS)), dim3(ROW_THREADS), 0, st, p);
    return launched();
}

int kqkv_rope_store(const kqkv_cache *cache, const kqkv_rope *rope, int T, const int32_t *pos, int64_t pos_stride,
                    const int32_t *slots, int q_heads, const float *q, int64_t ldq, float *q_out, int64_t ldq_out,
                    const float *k, int64_t ldk, const float *v, int64_t ldv, void *stream) {
    int r = cache_check(cache);
    if (r) return r;
    if (T < 0 || T >= (1 << 23) || q_heads < 0 || q_heads > 1024) return KQ_ERR_SHAPE;
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
    Rows x = {q, k, v, q_out, slots, ldq, ldq_out, ldk, ldv, q_heads, T, 1, k ? v_workgroups(cache, T) : 0, 0};
    const int lanes = cache->head_dim / 8, a_wg = 64 / lanes * STORE_WAVES, rows = q_heads + (k ? cache->kv_heads : 0);
    x.lanes_magic = (u32)((65536 + lanes - 1) / lanes);
    const bool q8 = cache->type == KQKV_Q8_0;
    hipStream_t st = (hipStream_t)stream;
    const Cache c = cache_args(cache);
    if (ra.pairs % 4 == 0) {
        // up to about 4 work-groups a compute unit, no more than a wave's rows each
        x.split = std::max(1, std::min((rows + a_wg - 1) / a_wg, 1024 / T));
        hipLaunchKernelGGL(q8 ? rope_store_kernel<true> : rope_store_kernel<false>, dim3((unsigned)(x.v_wgs + T * x.split)),
                           dim3(STORE_THREADS), 0, st, c, ra, x);
    } else {
        hipLaunchKernelGGL(q8 ? rope_store_any_kernel<true> : rope_store_any_kernel<false>, dim3((unsigned)(x.v_wgs + T)),
                           dim3(STORE_THREADS), 0, st, c, ra, x);
    }
    return launched();
}

int kqkv_load(const kqkv_cache *cache, int T, const int32_t *slots, float *k, float *v, void *stream) {
    const int r = cache_check(cache);
    if (r) return r;
    if (T < 0 || T >= (1 << 23)) return KQ_ERR_SHAPE;
    if (T == 0 || (!k && !v)) return KQ_OK;
    if (!slots) return KQ_ERR_NULL;
    if (!aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16)) return KQ_ERR_ALIGN;
    if (device_check()) return KQ_ERR_DEVICE;
    const int v_wgs = v ? v_workgroups(cache, T) : 0;
    hipLaunchKernelGGL(cache->type == KQKV_Q8_0 ? load_kernel<true> : load_kernel<false>, dim3((unsigned)(v_wgs + (k ? T : 0))),
                       dim3(STORE_THREADS), 0, (hipStream_t)stream, cache_args(cache), slots, T, k, v, v_wgs);
    return launched();
}

} // extern "C"
