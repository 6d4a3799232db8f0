// kq_attn.hip -- kqkv_attn of include/kqkv.h: argument checks and how the work
// is split.  The kernels are in kq_attn.h, instantiated per head size in
// kq_attn_inst.hip.
#include "kq_attn.h"

#include <cmath>

using namespace kq;
using namespace kq::kv;

// Contexts past this (half of the last-level cache) are not there any more when they are read again, another layer's
// having been read in between: where no two work-groups or waves share a line (up to 16 rows a kv head), lines are then
// read with the non-temporal hint (three caches in turn: one request of 131072 fp16 tokens 103 -> 90 us, 32 of 1024 27.7
// -> 23.9, 64 of up to 32768 Q8_0 tokens 310 -> 287; smaller ones that stay even or slower, 24 with a window of 1000 and
// heads of 64 15.1 -> 16.5).
constexpr double KEPT_BYTES = 128e6;

// The split of a call.  Returns the row tiles a wave.  (Measured with 64 query and 8 kv heads of 128 where nothing else is
// said; heads of other sizes and numbers follow the same rules.)
//  * Rows: up to 16 are one row tile; more, two tiles a wave (heads of up to 128) and up to 64 rows a work-group, whose
//    four waves share the rows first, then the keys (8 rows of 8 requests of 4096 fp16 tokens: one tile a wave 55 us, two
//    45).
//  * A piece has at least min_tiles tiles.  A work-group costs about 6 us beside its tiles (a chain of dependent loads,
//    the join of its waves) and a cut one its share of a second launch, so contexts are cut past 16 tiles where there
//    are few work-groups (8 where a tile is heavy), past 48 where requests and heads alone make one per compute unit.
//    Uncut against cut, fp16, 64 query and 8 kv heads of 128: one request of 512 tokens 8.8 us against 10.1, of 1024
//    13.2 against 10.2 (in pieces of 4; of 8 11.2); 8 of 512 10.5 against 12.5; 20 of 1024 17.5 against 23.4; 56 of 1536
//    57 against 72, 56 of 64 to 1536 35 against 41, 40 of them 34 against 30; 8 rows of one request of 512 20 against 17.
//  * Where it leaves each request two pieces or more on average, as many pieces as work-groups run at once and no more
//    (3 on each of 256 compute units, by their registers; with 30 % more, one request of 131072 tokens 113 us instead of
//    94, 8 rows of 8 requests of 4096 55 instead of 45).  Larger batches take up to four times that, 64 tiles a piece, so
//    that the requests' lengths even out (64 requests of up to 16384 fp16 tokens 318 us, in one round 322).  Contexts of up
//    to 256 tiles do so past 1.5 pieces only (64 requests of 8192 fp16 tokens: 96 pieces a head 325 us, 160 362; of up to
//    8192 89 and 91), but not rows of two tiles a wave (40 requests of 4096 Q8_0 tokens and 8 rows: 64 pieces 211 us, 104
//    166).
static int attn_split(const kqkv_cache *c, int B, int max_q, int64_t max_ctx, int q_heads, int window, Attn *a) {
    a->group = q_heads / c->kv_heads;
    a->rows_cap = a->group * max_q;
    const int rt = a->rows_cap <= 16 || c->head_dim > 32 * TWO_TILES_NB ? 1 : 2;
    a->row_waves = a->rows_cap <= 16 * rt ? 1 : rt == 2 || a->rows_cap <= 32 ? 2 : 4;
    auto magic = [](int d) { return d == 1 ? 0u : (u32)(((1ull << 32) + d - 1) / d); };
    a->group_magic = magic(a->group);
    a->gp_magic = magic(c->page_tokens / 16);
    const int wg_rows = 16 * rt * a->row_waves, groups = (a->rows_cap + wg_rows - 1) / wg_rows;
    if (window) max_ctx = std::min<int64_t>(max_ctx, (int64_t)window + max_q + 2 * TILE);
    const int64_t tiles = (max_ctx + TILE - 1) / TILE, base = (int64_t)B * c->kv_heads * groups;
    a->min_tiles = base < 32 ? 4 : base < 256 ? 8 : 32;
    const int64_t each = (int64_t)c->kv_heads * groups, at_once = 256 * ATTN_OCCUPANCY(c->head_dim / 32, rt);
    const int64_t whole = base < 32 && rt * c->head_dim > 128 ? 8 : base < 160 ? 16 : base < 256 ? 32 : 48;
    const int64_t most = tiles <= whole ? B : B * ((tiles + a->min_tiles - 1) / a->min_tiles);
    const int64_t items = 2 * (at_once / each) >= (rt == 1 && tiles <= 256 ? 3 : 4) * B ? at_once / each
                                                  : B + std::max<int64_t>(1, std::max(at_once, std::min(base * tiles / 64, 4 * at_once)) / each);
    a->items = (int)std::min(most, items);
    return rt;
}

// The pieces' unnormalised outputs with their m and l, then the requests'
// pieces (a.info).
static size_t part_bytes(const kqkv_cache *c, const Attn &a, int q_heads, int max_q) {
    return (size_t)a.items * q_heads * max_q * (c->head_dim + 4) * sizeof(float);
}

static int attn_shape(const kqkv_cache *cache, int B, int max_q, int64_t max_ctx, int q_heads) {
    if (B < 1 || B > 4096) return KQ_ERR_SHAPE;
    if (max_q < 1 || max_q > 8) return KQ_ERR_M;
    if (max_ctx < 1 || max_ctx > INT32_MAX) return KQ_ERR_SHAPE;
    if (q_heads < 1 || q_heads > 1024 || q_heads % cache->kv_heads) return KQ_ERR_SHAPE;
    if ((int64_t)B * q_heads * max_q >= (1 << 24)) return KQ_ERR_SHAPE;
    return KQ_OK;
}

extern "C" {

size_t kqkv_attn_workspace_bytes(const kqkv_cache *cache, int B, int max_q, int64_t max_ctx, int q_heads) {
    if (!cache || cache_limits(cache->type, cache->kv_heads, cache->head_dim, cache->page_tokens)) return 0;
    if (attn_shape(cache, B, max_q, max_ctx, q_heads)) return 0;
    Attn a;
    attn_split(cache, B, max_q, max_ctx, q_heads, 0, &a);
    return a.items <= B ? 0 : part_bytes(cache, a, q_heads, max_q) + (size_t)B * sizeof(int4);
}

int kqkv_attn(const kqkv_cache *cache, int B, int max_q, int64_t max_ctx, const int32_t *ctx_len,
              const int32_t *seq_start, const int32_t *table, int64_t table_stride, int q_heads, int T, const float *q,
              int64_t ldq, float scale, int window, float *out, int64_t ldo, void *workspace, size_t workspace_bytes,
              int32_t *err_flag, void *stream) {
    int r = cache_check(cache);
    if (r || (r = attn_shape(cache, B, max_q, max_ctx, q_heads))) return r;
    if (table_stride < 1 || table_stride > (1 << 24) || T < 0 || T >= (1 << 24)) return KQ_ERR_SHAPE;
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
    Attn a;
    const int rt = attn_split(cache, B, max_q, max_ctx, q_heads, window, &a);
    a.ctx_len = ctx_len;
    a.seq_start = seq_start;
    a.table = table;
    a.q = q;
    a.out = out;
    a.part = (float *)workspace;
    a.info = (int4 *)((char *)workspace + part_bytes(cache, a, q_heads, max_q));
    a.err = err_flag;
    a.stride = table_stride;
    a.ldq = ldq;
    a.ldo = ldo;
    a.B = B;
    a.T = T;
    a.max_q = max_q;
    a.window = window;
    a.scale = (float)(scale * 1.4426950408889634);
    const bool q8 = cache->type == KQKV_Q8_0;
    const Cache c = cache_args(cache);
    const int64_t seen = window ? std::min<int64_t>(max_ctx, (int64_t)window + max_q) : max_ctx;
    const bool nt = rt == 1 && a.row_waves == 1 && (double)B * seen * 2 * c.page_bytes / c.page_tokens > KEPT_BYTES;
    hipStream_t st = (hipStream_t)stream;
    switch (cache->head_dim / 32) {
    case 1: return launch_attn<1>(q8, nt, rt, c, a, st);
    case 2: return launch_attn<2>(q8, nt, rt, c, a, st);
    case 3: return launch_attn<3>(q8, nt, rt, c, a, st);
    case 4: return launch_attn<4>(q8, nt, rt, c, a, st);
    case 5: return launch_attn<5>(q8, nt, rt, c, a, st);
    case 6: return launch_attn<6>(q8, nt, rt, c, a, st);
    case 7: return launch_attn<7>(q8, nt, rt, c, a, st);
    default: return launch_attn<8>(q8, nt, rt, c, a, st);
    }
}

} // extern "C"
