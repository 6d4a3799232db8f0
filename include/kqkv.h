/*
 * kqkv.h -- the paged key-value cache beside the dequant-GEMV calls of
 * kqgemv.h, for AMD Instinct MI355X (gfx950): what a decode or verify step
 * does between a layer's q, k, v projections and its output projection.
 *
 *   kqkv_plan        once per step: pages taken and given back, and the slots,
 *                    positions and row offsets of the step's new tokens
 *   kqkv_rope_store  once per layer: rotary positions on q and k, and k and v
 *                    into the cache
 *   kqkv_attn        once per layer: each request's 1..8 new tokens over its
 *                    cached keys and values
 *   kqkv_load        cached tokens back as fp32
 *
 * (The Kortex summary, "Out-of-core LLM inference engine written from scratch
 * in Rust", section Approach, names a packed f16 key-value cache next to its
 * fused dequant-matmul kernels, and checks several draft positions per pass;
 * GGUF engines also keep the cache in Q8_0 blocks.)
 *
 * Activations are fp32 as in kqgemv.h: q, k and v are what kq_qgemv_multi
 * writes, the attention's output is what kq_qgemv reads.
 *
 * The cache.  K and V are two arrays of n_pages pages.  A page holds
 * page_tokens (P) consecutive tokens of one request for every kv head, head
 * after head.  Of one head (D = head_dim) it holds
 *   K: the tokens' rows, element (t, d) at t * D + d
 *   V: groups of 16 tokens, transposed: (t, d) at (t / 16) * 16 * D + d * 16 + t % 16
 * as fp16 (KQKV_F16), or as int8 quants (KQKV_Q8_0) that are followed by their
 * fp16 scales, one per token and 32 elements, for K and V alike at
 * (t / 16) * (D / 32) * 16 + (d / 32) * 16 + t % 16; a value is scale * quant, and
 * no scale is negative.
 * Token t of page p is slot p * P + t.  Memory that holds no token may hold
 * anything, NaN included.
 *
 * Conventions are those of kqgemv.h: device pointers owned by the caller, no
 * allocation, no synchronisation, asynchronous on `stream` of the current
 * device, negative kq_status for argument errors before any HIP call.  Every
 * call can be captured into a graph; what a replay computes follows the
 * contents of the device arrays at that time.  Calls on different streams run
 * side by side when they write different memory (each needs its own
 * workspace).  Results do not depend on timing, except where two rows of one call
 * name the same slot.  All int32 arrays 4-byte aligned;
 * fp32 rows 16-byte aligned with strides that are multiples of 4 floats.
 *
 * Device-side checks.  Lengths, pages and slots are read on the device only.
 * A value that would leave the arrays is never followed: where a call has an
 * err_flag (NULL or a device int32) it is set to 1 (never cleared), and the
 * call does what it says below.
 */
#ifndef KQKV_H
#define KQKV_H

#include <stddef.h>
#include <stdint.h>

#include "kqgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Cache element formats, by their GGUF type ids. */
enum { KQKV_F16 = 1, KQKV_Q8_0 = 8 };

typedef struct kqkv_cache {
    int type;            /* KQKV_F16 or KQKV_Q8_0                           */
    int kv_heads;        /* 1..1024                                         */
    int head_dim;        /* a multiple of 32, 32..256                       */
    int page_tokens;     /* a multiple of 16, 16..256                       */
    int64_t n_pages;     /* 1 <= n_pages, n_pages * page_tokens < 2^31      */
    void *k, *v;         /* n_pages * kqkv_page_bytes each, 16-B aligned    */
} kqkv_cache;

/* Bytes of one page of K (or of V): kv_heads * P * D * 2 (fp16), or
 * kv_heads * P * D * 17 / 16 (Q8_0).  A negative kq_status for sizes outside
 * the limits above.  Host-only. */
int64_t kqkv_page_bytes(int type, int kv_heads, int head_dim, int page_tokens);

/* The pages and slots of one step, from the requests' lengths.
 *
 * Request b (of B) has ctx_len[b] cached tokens and holds the pages
 * table[b][0 .. held[b]).  It gets new_len[b] >= 0 new tokens, for which it
 * takes max(0, ceil((ctx_len + new_len) / P) - held) pages; new_len[b] < 0
 * ends it: it gives its pages back and its length becomes 0.  (A request may
 * hold more pages than its length needs, as after a verify pass whose tokens
 * were not all accepted: set ctx_len back and plan the next step.)
 * free_pages[0 .. *n_free) is the list of pages nobody holds, room for n_pages
 * entries.  First the ended requests' pages go on top of it, in order of
 * request and page; then the other requests, in order, take theirs from the
 * top.
 *   table      [B] rows of table_stride entries; the new pages' entries are
 *              written, all others are left
 *   held_out   [B] pages held after the step (may be held)
 *   n_free_out list length after the step (may be n_free)
 *   ctx_out    [B] lengths with the new tokens (may be ctx_len)
 *   seq_start  [B + 1] first row of each request's new tokens: rows
 *              seq_start[b] .. seq_start[b + 1], in order
 *   slots, pos [T] slot and position (ctx_len + i) of row t; -1 and 0 for rows
 *              behind the last request's (and slot -1 where the table names a
 *              page outside [0, n_pages))
 * All or nothing: when the pages do not suffice, a request would need more than
 * table_stride pages, the new tokens number more than T, or a length, held or
 * n_free is out of range, then *err_flag = 1, slots are -1, pos and seq_start
 * 0, lengths, held and n_free come out unchanged, table and free_pages are left.
 * With in-place arguments (held_out == held, ...) the step is taken once per
 * call; with separate ones the call may be repeated with the same result.
 * 1 <= B <= 65536, 0 <= T < 2^23, 1 <= table_stride <= 2^24, page_tokens and
 * n_pages as in a cache.  slots and pos may be NULL when T is 0. */
int kqkv_plan(int B, const int32_t *ctx_len, const int32_t *new_len, int page_tokens,
              int32_t *table, int64_t table_stride, const int32_t *held, int32_t *held_out,
              int32_t *free_pages, int64_t n_pages, const int32_t *n_free, int32_t *n_free_out,
              int T, int32_t *slots, int32_t *pos, int32_t *seq_start, int32_t *ctx_out,
              int32_t *err_flag, void *stream);

/* Which two elements of a head rotate together, for pair i < rot_dims / 2. */
enum {
    KQKV_ROPE_HALVES = 0,    /* i and i + rot_dims / 2 */
    KQKV_ROPE_PAIRS = 1      /* 2i and 2i + 1          */
};

/* Rotary positions.  Pair i = (a, b) of a token at positions pos[axis] turns
 * by the angle t = pos[axis(i)] / (base^(2i / rot_dims) * freq_factors[i]):
 * (a cos t - b sin t, a sin t + b cos t).  The first sections[0] pairs take
 * axis 0, the next sections[1] axis 1, ... (images and video: time, height,
 * width); with one axis, sections[0] = rot_dims / 2.  Elements past rot_dims
 * do not turn.  Angles and rotation are computed in 64 bits (the angle's
 * error is about pos * 2^-52) and rounded once to fp32. */
typedef struct kqkv_rope {
    int style;                    /* KQKV_ROPE_*                                */
    int rot_dims;                 /* even, 2..head_dim                          */
    float base;                   /* > 0, finite                                */
    int n_axes;                   /* 1..4                                       */
    int sections[4];              /* pairs of each axis, >= 0, sum rot_dims / 2 */
    const float *freq_factors;    /* NULL (all 1) or device [rot_dims / 2]      */
} kqkv_rope;

/* Rotary positions on q and k, and k and v into the cache, for T tokens.
 *   pos    [n_axes] rows of pos_stride int32, one position per token
 *   slots  [T] cache slot of each token; a token whose slot is outside the
 *          cache (-1 for padding) is not stored (its q is still rotated)
 *   q      [T] rows of q_heads * head_dim fp32, row stride ldq; q_out the same
 *          with stride ldq_out; q_out may be q (with ldq_out == ldq) but not
 *          overlap it otherwise.  q_heads 0: no q
 *   k, v   [T] rows of kv_heads * head_dim fp32, strides ldk and ldv; left as
 *          they are.  Both NULL: nothing is stored
 * rope NULL: nothing turns (q_heads must be 0).  fp16 values are rounded to
 * nearest (beyond the fp16 range: infinities).  A Q8_0 block of 32 values x has
 * the scale s = fp16(max|x| * (1 / 127)), reciprocal and product rounded to
 * fp32, at most 65504, and the quants rint(x / s), -127..127 (0 when s is 0); a
 * block with an infinity or a NaN gets a NaN scale.  (GGUF's quantiser divides by
 * 127 and makes the quants from that quotient unrounded: about one scale in 10^6
 * is its neighbour, and quants near a half step differ.)  When two tokens name
 * the same slot, either's values or a mixture stay there.  0 <= T < 2^23,
 * q_heads <= 1024. */
int kqkv_rope_store(const kqkv_cache *cache, const kqkv_rope *rope, int T, const int32_t *pos, int64_t pos_stride,
                    const int32_t *slots, int q_heads, const float *q, int64_t ldq, float *q_out, int64_t ldq_out,
                    const float *k, int64_t ldk, const float *v, int64_t ldv, void *stream);

/* Cached tokens as fp32: k[t], v[t] = rows of kv_heads * head_dim values of
 * slot slots[t] (contiguous rows; either may be NULL).  Exact for both formats.
 * Rows whose slot is outside the cache are left as they are.  0 <= T < 2^23. */
int kqkv_load(const kqkv_cache *cache, int T, const int32_t *slots, float *k, float *v, void *stream);

/* Workspace bytes of kqkv_attn for such a call (0 on invalid sizes; may be 0
 * where nothing is split). */
size_t kqkv_attn_workspace_bytes(const kqkv_cache *cache, int B, int max_q, int64_t max_ctx, int q_heads);

/* Attention of each request's new tokens over its cached tokens.
 *
 * Request b's new tokens are the rows seq_start[b] .. seq_start[b + 1] of q and
 * out, the last ones of its ctx_len[b] cached tokens (kqkv_plan's seq_start
 * and ctx_out; their k and v are in the cache).  Row j of n sits at position
 * p = ctx_len[b] - n + j and, for each query head h with the keys and values of
 * kv head h / (q_heads / kv_heads),
 *   out = sum_i w_i v_i / sum_i w_i,  w_i = exp(scale * q . k_i),
 * over the tokens i <= p, and with window > 0 those with i > p - window.  A
 * row that no token remains for is 0.
 *   table      [B] rows of table_stride pages; token i is in page
 *              table[b][i / P]
 *   max_q      rows of the longest request, 1..8 (one new token, or the
 *              positions of a verify pass); rows of a request past max_q are
 *              left, and *err_flag is set
 *   max_ctx    the longest context expected, 1 .. 2^31 - 1: it sets how the
 *              work is split (a longer one is computed all the same, slowly
 *              when max_ctx was short)
 *   q, out     [T] rows of q_heads * head_dim fp32, strides ldq and ldo; out
 *              must not overlap q.  Rows that belong to no request are left;
 *              rows past T are never touched
 *   workspace  kqkv_attn_workspace_bytes, 16-B aligned; scratch that needs no
 *              preparation and keeps nothing between calls
 * A page outside [0, n_pages), or a length past table_stride * P (or 2^31 - 64),
 * takes its tokens out of the sum and sets *err_flag; a negative length counts as
 * 0.
 * Accumulation is fp32; q and the weights enter the matrix instructions as two
 * fp16 limbs (22 bits, weights no finer than 2^-31 of their row's largest), the
 * cached values as they are.  |scale * q| is to stay below 2^100.  What a row does
 * not see never reaches it, whatever it holds; infinities and NaN in a key or
 * value that it sees, and values that a Q8_0 cache holds past the fp16 range
 * (65504), give infinities or NaN (an infinite key also where its weight would be
 * 0).  Reruns are bit-identical; a request's bits may depend on the other
 * requests' lengths (they set where its tokens are split).  1 <= B <= 4096,
 * q_heads a multiple of kv_heads, at most 1024, B * q_heads * max_q < 2^24,
 * 0 <= T < 2^24, window >= 0, scale finite. */
int kqkv_attn(const kqkv_cache *cache, int B, int max_q, int64_t max_ctx, const int32_t *ctx_len,
              const int32_t *seq_start, const int32_t *table, int64_t table_stride, int q_heads, int T,
              const float *q, int64_t ldq, float scale, int window, float *out, int64_t ldo,
              void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KQKV_H */
