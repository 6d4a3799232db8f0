/*
 * kqstep.h -- what a decode or verify step does beside the dequant-GEMV calls
 * of kqgemv.h and the paged cache of kqkv.h, for AMD Instinct MI355X (gfx950):
 *
 *   kqstep_norm     the residual's addition and the root-mean-square norm,
 *                   of a token's row or of each of its heads
 *   kqstep_moe      a whole mixture-of-experts layer: router, choice of the
 *                   experts, their gate and up products, activation, down
 *                   products and weighted sum
 *   kqstep_sample   a token for each row of logits
 *
 * (The Kortex article, "Kortex: Streaming 70B Models on Consumer GPUs", and the
 * RunNburn post, "RunNburn - Run a 295B Moe from a 98GB GGUF on a 64GB RAM
 * Desktop", decode whole models, mixture-of-experts ones among them, with
 * greedy and temperature sampling; their pages print no kernel of these.)
 *
 * Activations are fp32 as in kqgemv.h: what kqstep_norm writes, kq_qgemv_multi
 * and kqstep_moe read; what kq_qgemv writes for the output matrix,
 * kqstep_sample reads.
 *
 * Conventions are those of kqgemv.h and kqkv.h: device pointers owned by the
 * caller, no allocation, no synchronisation, asynchronous on `stream` of the
 * current device, negative kq_status for argument errors before any HIP call.
 * Every call can be captured into a graph; what a replay computes follows the
 * contents of the device arrays at that time.  Calls on different streams run
 * side by side when they write different memory (each needs its own
 * workspace).  A workspace is scratch that needs no preparation and keeps
 * nothing between calls.  Reruns are bit-identical, and a token's (or row's)
 * results do not depend on the other tokens of its call or on their number.  Rows of fp32 are
 * 16-byte aligned with strides that are multiples of 4 floats (kqstep_sample's
 * logits: any); int32 and float arrays 4-byte aligned, workspaces 16-byte.
 */
#ifndef KQSTEP_H
#define KQSTEP_H

#include <stddef.h>
#include <stdint.h>

#include "kqgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Residual addition and root-mean-square norm.
 *
 * A token's row is `heads` parts of n elements, each normed by itself (heads 1:
 * the whole row; heads > 1: the query or key heads of a row of projections).
 * For every part,
 *   h = x + add                          (add NULL: h = x)
 *   y = h * weight / sqrt(sum(h * h) / n + eps)
 * h is rounded to fp32; the sum of squares, the root and the products are in 64
 * bits, and y is rounded once.
 *   x, add   [T] rows of heads * n fp32, strides ldx and ldadd
 *   sum      h, stride ldsum; NULL: not written.  Needs add
 *   weight   [n] fp32, the same for every head, 16-B aligned; NULL: all 1
 *   y        stride ldy; NULL: not written
 *   y8       y in Q8_0 blocks: T consecutive rows of
 *            kq_row_bytes(KQ_TYPE_Q8_0, heads * n) bytes, 16-B aligned, which
 *            kq_dequant reads; NULL: not written.  Needs n a multiple of 32.
 *            Blocks are made as kqkv_rope_store makes the cache's (scale
 *            fp16(max|y| * (1 / 127)), at most 65504, nearest quants of that
 *            scale; NaN scale with an infinity or a NaN in the block)
 * One of y and y8 has to be given.  sum and y may each be x or add (with the
 * same stride); they must not overlap anything otherwise.  Rows hold what the
 * arithmetic gives for infinities and NaN; a row of zeros is 0 for eps > 0.
 * 0 <= T < 2^23, 1 <= heads <= 1024, n a multiple of 4, heads * n <= 2^20,
 * T * heads < 2^31, eps >= 0 and finite. */
int kqstep_norm(int T, int heads, int n, const float *x, int64_t ldx, const float *add, int64_t ldadd, float *sum,
                int64_t ldsum, const float *weight, float eps, float *y, int64_t ldy, void *y8, void *stream);

/* How a router's logits become the experts' scores. */
enum {
    KQSTEP_SOFTMAX = 0,     /* exp(l) / sum over all experts of exp(l) */
    KQSTEP_SIGMOID = 1      /* 1 / (1 + exp(-l))                       */
};

/* Activation of the gate. */
enum {
    KQSTEP_SILU = 0,        /* g / (1 + exp(-g))                                       */
    KQSTEP_GELU = 1         /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2       */
};

/* A layer's weights and its routing. */
typedef struct kqstep_moe_layer {
    int E;                  /* experts, 1..1024                                     */
    int k;                  /* experts of a token, 1..16, <= E                      */
    int64_t hidden, inner;  /* row sizes, each a positive multiple of its types'
                               block size, <= 2^20                                  */
    int gate_type;          /* block format of gate and up (a kq_type)              */
    int down_type;          /* ... and of down                                      */
    const void *gate, *up;  /* E matrices of inner rows of hidden weights, as
                               kq_qmoe_gemv takes them (16-B aligned)               */
    const void *down;       /* E matrices of hidden rows of inner weights           */
    const float *router;    /* [E][hidden] fp32, 16-B aligned                       */
    const float *bias;      /* [E] added to the scores for the choice alone, or NULL */
    int score;              /* KQSTEP_SOFTMAX or KQSTEP_SIGMOID                     */
    int renorm;             /* nonzero: a token's weights are divided by their sum  */
    float scale;            /* factor of the weights, finite                        */
    int act;                /* KQSTEP_SILU or KQSTEP_GELU                           */
} kqstep_moe_layer;

/* Workspace bytes of kqstep_moe for T tokens; 0 on invalid sizes. */
size_t kqstep_moe_workspace_bytes(const kqstep_moe_layer *layer, int T);

/* A mixture-of-experts layer for 1 <= T <= 8 tokens.
 *
 *   l = router . x, scores s of l; the token's experts e_1 .. e_k are those of
 *   the largest l (with a bias: s + bias), descending, ties to the lower expert;
 *   p_j = s(e_j) * scale, with renorm s(e_j) * scale / sum_j s(e_j);
 *   y = add + sum_j p_j down[e_j] . (act(gate[e_j] . x) * (up[e_j] . x))
 *
 * Logits, scores and weights are computed in 64 bits (so that experts whose
 * logits differ by an fp32 rounding are not mistaken for each other), the weights
 * rounded once; the products as in kq_qgemv, in fp32, each within 1e-4 *
 * sum|w*x| + 1e-6 of the exact one.
 *   x, add, y  [T] rows of `hidden` fp32, strides ldx, ldadd, ldy.  add NULL: 0.
 *              y may be add (with the same stride) and must not overlap x
 *   ids        [T][k] int32 the chosen experts, or NULL
 *   weights    [T][k] fp32 p, or NULL
 *   workspace  kqstep_moe_workspace_bytes
 * A NaN logit (or score with its bias) counts as the lowest; a token with an
 * infinity or a NaN in x, or whose scores sum to 0, gets what the arithmetic
 * gives (its ids stay valid). */
int kqstep_moe(const kqstep_moe_layer *layer, int T, const float *x, int64_t ldx, const float *add, int64_t ldadd,
               float *y, int64_t ldy, int32_t *ids, float *weights, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of kqstep_sample; 0 on invalid sizes. */
size_t kqstep_sample_workspace_bytes(int M, int64_t V);

/* One token for each of M rows of V logits.
 *
 * With the row's temperature t > 0 a token's weight is w = exp((l - max l) / t).
 * Tokens stand in the order of their logits, descending, ties by index; a
 * leading part of that order is kept, the shortest that any of these leaves (the
 * first token always stays):
 *   top_k  its first top_k tokens (<= 0: all)
 *   top_p  the shortest leading part whose weight is at least top_p of the
 *          weight that top_k leaves (>= 1: all)
 *   min_p  the tokens with w >= min_p
 * The token is the lowest index for which the kept weights up to and with it, in
 * the order of the indices, sum to more than u times all kept weights; u is a
 * given random number in [0, 1).  t <= 0 (or NaN): the first token of the order.
 * A logit that is NaN counts as -infinity; a token at -infinity is never taken;
 * where a row has no other, its token is -1 and its probability 0.
 *   logits       [M] rows of V fp32, ld >= V apart, 4-byte aligned
 *   temperature, top_p, min_p, u  [M] fp32; top_k [M] int32.  NULL: temperature
 *                1, all tokens kept; u is always needed (outside [0, 1): the nearest)
 *   tokens       [M] int32
 *   probs        [M] fp32 the token's part of the kept weight, or NULL
 *   workspace    kqstep_sample_workspace_bytes
 * Weights are computed in 64 bits and rounded to 36 of mantissa, however far from 0
 * the logits lie; those 64 octaves below the row's largest count as 0 (from 63 3/4
 * on some of them).  They are summed as integers, and such sums in 64 bits in a fixed
 * order: the kept weight is off by less than 2^-35 of itself.
 * 0 <= M <= 65536, 1 <= V <= 2^20. */
int kqstep_sample(int M, int64_t V, const float *logits, int64_t ld, const float *temperature, const int32_t *top_k,
                  const float *top_p, const float *min_p, const float *u, int32_t *tokens, float *probs, void *workspace,
                  size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KQSTEP_H */
