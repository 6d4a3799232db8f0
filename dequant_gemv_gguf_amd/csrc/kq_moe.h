// kq_moe.h -- what the translation units of kqstep_moe share: a call as its
// kernels see it, and the launchers of one block format (kq_moe_inst.hip, one
// object per format).
#pragma once

#include "kq_step.h"

namespace kq {
namespace step {

constexpr int MOE_TOKENS = 8, MOE_EXPERTS = 1024, MOE_SLOTS = 16;

struct Moe {
    const float *x, *add, *router, *bias;
    const uint8_t *gate, *up, *down;
    float *y;
    int32_t *ids;               // [T][k], the caller's or scratch, as weights
    float *weights;             // [T][k]
    double *logits;             // [T][E] scratch
    float *inner;               // [T][k][inner] scratch
    int64_t ldx, ldadd, ldy;
    int64_t gate_bytes, down_bytes;     // of one row
    double scale;
    int E, k, hidden, n_inner, T;
    int score, renorm, act;
};

template <int T> int launch_gate_up(const Moe &a, hipStream_t st);
template <int T> int launch_down(const Moe &a, hipStream_t st);

#define KQ_MOE_LAUNCHERS(X, T)                        \
    X int launch_gate_up<T>(const Moe &, hipStream_t); \
    X int launch_down<T>(const Moe &, hipStream_t);

} // namespace step
} // namespace kq
