// kq_attn.hip -- attention of a few new tokens per request over the paged
// cache (kqkv_attn in include/kqkv.h).
#include "kq_kv.h"

#include <cmath>

namespace kq {
namespace kv {

struct Attn {
    const int32_t *ctx_len, *seq_start, *table;
    const float *q;
    float *out;
    int32_t *err;
    int64_t stride, ldq, ldo;
    int B, T, max_q, group, window;
    float scale;
};

// One wave per row and query head: keys one after another, the running
// maximum and sum of the softmax.
template <bool Q8>
__global__ __launch_bounds__(64) void attn_kernel(Cache c, Attn a) {
    const int b = blockIdx.x / a.max_q, j = blockIdx.x % a.max_q, h = blockIdx.y, lane = threadIdx.x;
    const int first = a.seq_start[b], n = a.seq_start[b + 1] - first;
    const int64_t row = (int64_t)first + j;
    if (j >= n || row < 0 || row >= a.T) return;
    const int kh = h / a.group;
    const int64_t ctx = max(a.ctx_len[b], 0), room = a.stride * c.page_tokens;
    const int64_t p = ctx - n + j;
    if (ctx > room && lane == 0 && a.err) a.err[0] = 1;
    const int64_t end = min(p + 1, room), begin = a.window ? max((int64_t)0, p - a.window + 1) : 0;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    for (int i = 0; i < 4; ++i)
        q[i] = lane + 64 * i < c.dim ? a.q[row * a.ldq + (int64_t)h * c.dim + lane + 64 * i] : 0.f;
    for (int64_t t = begin; t < end; ++t) {
        const u32 page = (u32)a.table[b * a.stride + t / c.page_tokens], at = (u32)(t % c.page_tokens);
        if (page >= c.n_pages) {
            if (lane == 0 && a.err) a.err[0] = 1;
            continue;
        }
        const int64_t off = page * c.page_bytes + (int64_t)kh * c.head_bytes;
        float s = 0.f, v[4];
        for (int i = 0; i < 4; ++i) {
            const u32 d = lane + 64 * i;
            v[i] = 0.f;
            if (d >= (u32)c.dim) continue;
            const u32 ki = k_at(at, d, c.dim), vi = v_at(at, d, c.dim);
            if (Q8) {
                const u32 si = scale_at(at, d >> 5, c.dim), tail = c.page_tokens * c.dim;
                s = fmaf(q[i], (float)((const _Float16 *)(c.k + off + tail))[si] * (float)((const int8_t *)(c.k + off))[ki], s);
                v[i] = (float)((const _Float16 *)(c.v + off + tail))[si] * (float)((const int8_t *)(c.v + off))[vi];
            } else {
                s = fmaf(q[i], (float)((const _Float16 *)(c.k + off))[ki], s);
                v[i] = (float)((const _Float16 *)(c.v + off))[vi];
            }
        }
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
        s *= a.scale;
        const float top = fmaxf(m, s), keep = m == top ? 1.f : expf(m - top), w = expf(s - top);
        l = l * keep + w;
        for (int i = 0; i < 4; ++i) o[i] = o[i] * keep + w * v[i];
        m = top;
    }
    for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < c.dim) a.out[row * a.ldo + (int64_t)h * c.dim + lane + 64 * i] = l == 0.f ? 0.f : o[i] / l;
}

} // namespace kv
} // namespace kq

using namespace kq;
using namespace kq::kv;

static int attn_shape(const kqkv_cache *cache, int B, int max_q, int64_t max_ctx, int q_heads) {
    if (B < 1 || B > 4096) return KQ_ERR_SHAPE;
    if (max_q < 1 || max_q > 8) return KQ_ERR_M;
    if (max_ctx < 1 || max_ctx > INT32_MAX) return KQ_ERR_SHAPE;
    if (q_heads < 1 || q_heads > 1024 || q_heads % cache->kv_heads) return KQ_ERR_SHAPE;
    return KQ_OK;
}

extern "C" {

size_t kqkv_attn_workspace_bytes(const kqkv_cache *cache, int B, int max_q, int64_t max_ctx, int q_heads) {
    if (!cache || cache_limits(cache->type, cache->kv_heads, cache->head_dim, cache->page_tokens)) return 0;
    if (attn_shape(cache, B, max_q, max_ctx, q_heads)) return 0;
    return 0;
}

int kqkv_attn(const kqkv_cache *cache, int B, int max_q, int64_t max_ctx, const int32_t *ctx_len,
              const int32_t *seq_start, const int32_t *table, int64_t table_stride, int q_heads, int T, const float *q,
              int64_t ldq, float scale, int window, float *out, int64_t ldo, void *workspace, size_t workspace_bytes,
              int32_t *err_flag, void *stream) {
    int r = cache_check(cache);
    if (r || (r = attn_shape(cache, B, max_q, max_ctx, q_heads))) return r;
    if (table_stride < 1 || table_stride > (1 << 24) || T < 0 || T >= (1 << 27)) return KQ_ERR_SHAPE;
    if (window < 0 || !std::isfinite(scale)) return KQ_ERR_ARG;
    if (T == 0) return KQ_OK;
    if (!ctx_len || !seq_start || !table) return KQ_ERR_NULL;
    if (!aligned(ctx_len, 4) || !aligned(seq_start, 4) || !aligned(table, 4) || !aligned(err_flag, 4)) return KQ_ERR_ALIGN;
    const int64_t n = (int64_t)q_heads * cache->head_dim;
    if ((r = rows_check(q, ldq, n)) || (r = rows_check(out, ldo, n))) return r;
    const size_t ws = kqkv_attn_workspace_bytes(cache, B, max_q, max_ctx, q_heads);
    if (ws && !workspace) return KQ_ERR_NULL;
    if (ws && !aligned(workspace, 16)) return KQ_ERR_ALIGN;
    if (workspace_bytes < ws) return KQ_ERR_SHAPE;
    if (device_check()) return KQ_ERR_DEVICE;
    const Attn a = {ctx_len, seq_start, table, q, out, err_flag, table_stride, ldq, ldo, B, T, max_q,
                    q_heads / cache->kv_heads, window, scale};
    hipStream_t st = (hipStream_t)stream;
    const dim3 grid(B * max_q, q_heads);
    if (cache->type == KQKV_F16) hipLaunchKernelGGL(attn_kernel<false>, grid, dim3(64), 0, st, cache_args(cache), a);
    else hipLaunchKernelGGL(attn_kernel<true>, grid, dim3(64), 0, st, cache_args(cache), a);
    return launched();
}

} // extern "C"
