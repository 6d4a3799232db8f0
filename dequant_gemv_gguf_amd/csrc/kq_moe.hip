// kq_moe.hip -- the router and the C ABI of kqstep_moe (include/kqstep.h).  The
// experts' products are in kq_moe_inst.hip.
#include "kq_moe.h"

#include <cmath>

namespace kq {
namespace step {

KQ_MOE_LAUNCHERS(extern template, T_Q4_0)
KQ_MOE_LAUNCHERS(extern template, T_Q8_0)
KQ_MOE_LAUNCHERS(extern template, T_Q2_K)
KQ_MOE_LAUNCHERS(extern template, T_Q3_K)
KQ_MOE_LAUNCHERS(extern template, T_Q4_K)
KQ_MOE_LAUNCHERS(extern template, T_Q5_K)
KQ_MOE_LAUNCHERS(extern template, T_Q6_K)

// Router.  Bound: the chain of a launch, one read and a reduction (the matrix
// is a few MB): 128 experts of 2048 and one token 2.9 us, of 160 of 5120 and three 5.
// A work-group an expert: products of fp32 values are exact in 64 bits, the sums'
// order does not depend on T.  (With 256 threads, one read more after the other, a
// layer of three tokens of 5120 took 85.2 us, with 512 84.3.)
constexpr int ROUTER_THREADS = 512;

// A work-group takes up to NT tokens: their rows are asked for together (past T: the
// last one's again).
template <int NT>
__global__ __launch_bounds__(ROUTER_THREADS) void router_kernel(const Moe a) {
    __shared__ double waves[NT][ROUTER_THREADS / 64];
    const int e = blockIdx.x, t0 = blockIdx.y * NT, tid = threadIdx.x;
    const float *w = a.router + (int64_t)e * a.hidden, *x[NT];
    double acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        x[t] = a.x + min(t0 + t, a.T - 1) * a.ldx;
        acc[t] = 0.0;
    }
    for (int i = 4 * tid; i < a.hidden; i += 4 * ROUTER_THREADS) {
        const f4 v = *(const f4 *)(w + i);
        f4 xs[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xs[t] = *(const f4 *)(x[t] + i);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t] = fma((double)v[j], (double)xs[t][j], acc[t]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const double s = sum_d<64>(acc[t]);
        if ((tid & 63) == 0) waves[t][tid >> 6] = s;
    }
    __syncthreads();
    if (tid < NT && t0 + tid < a.T) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < ROUTER_THREADS / 64; ++i) s += waves[tid][i];
        a.logits[(t0 + tid) * a.E + e] = s;
    }
}

template <int NT> static void launch_router(const Moe &a, hipStream_t st) {
    hipLaunchKernelGGL(router_kernel<NT>, dim3((unsigned)a.E, (unsigned)((a.T + NT - 1) / NT)), dim3(ROUTER_THREADS), 0, st, a);
}
// Tokens of a work-group: as few as two work-groups a compute unit leave.
static void launch_router(const Moe &a, hipStream_t st) {
    const int groups = std::max(1, 2 * cu_count() / a.E), n = (a.T + groups - 1) / groups;
    if (n <= 1) launch_router<1>(a, st);
    else if (n <= 2) launch_router<2>(a, st);
    else if (n <= 4) launch_router<4>(a, st);
    else launch_router<8>(a, st);
}

static int layer_check(const kqstep_moe_layer *l, int64_t *gate_bytes, int64_t *down_bytes) {
    if (!l) return KQ_ERR_NULL;
    int qk, nb, upb;
    if (l->E < 1 || l->E > MOE_EXPERTS || l->k < 1 || l->k > MOE_SLOTS || l->k > l->E) return KQ_ERR_ARG;
    if (fmt_of(l->gate_type, &qk, &nb, &upb)) return KQ_ERR_TYPE;
    if (l->hidden <= 0 || l->hidden % qk || l->hidden > (1 << 20)) return KQ_ERR_SHAPE;
    *gate_bytes = l->hidden / qk * nb;
    if (fmt_of(l->down_type, &qk, &nb, &upb)) return KQ_ERR_TYPE;
    if (l->inner <= 0 || l->inner % qk || l->inner > (1 << 20)) return KQ_ERR_SHAPE;
    *down_bytes = l->inner / qk * nb;
    return KQ_OK;
}

static size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

// The parts of a workspace: logits, inner rows, ids, weights.
struct MoeSpace { size_t inner, ids, weights, end; };
static MoeSpace moe_space(const kqstep_moe_layer *l, int T) {
    MoeSpace s;
    s.inner = round16((size_t)T * l->E * sizeof(double));
    s.ids = s.inner + round16((size_t)T * l->k * l->inner * sizeof(float));
    s.weights = s.ids + round16((size_t)T * l->k * sizeof(int32_t));
    s.end = s.weights + round16((size_t)T * l->k * sizeof(float));
    return s;
}

} // namespace step
} // namespace kq

using namespace kq;
using namespace kq::step;

extern "C" {

size_t kqstep_moe_workspace_bytes(const kqstep_moe_layer *layer, int T) {
    int64_t a, b;
    if (layer_check(layer, &a, &b) || T < 1 || T > MOE_TOKENS) return 0;
    return moe_space(layer, T).end;
}

int kqstep_moe(const kqstep_moe_layer *layer, int T, const float *x, int64_t ldx, const float *add, int64_t ldadd,
               float *y, int64_t ldy, int32_t *ids, float *weights, void *workspace, size_t workspace_bytes, void *stream) {
    int64_t gate_bytes, down_bytes;
    int r = layer_check(layer, &gate_bytes, &down_bytes);
    if (r) return r;
    if (layer->score != KQSTEP_SOFTMAX && layer->score != KQSTEP_SIGMOID) return KQ_ERR_ARG;
    if (layer->act != KQSTEP_SILU && layer->act != KQSTEP_GELU) return KQ_ERR_ARG;
    if (!std::isfinite(layer->scale)) return KQ_ERR_ARG;
    if (T < 1 || T > MOE_TOKENS) return KQ_ERR_M;
    if (!layer->gate || !layer->up || !layer->down || !layer->router || !workspace) return KQ_ERR_NULL;
    if (!aligned(layer->gate, 16) || !aligned(layer->up, 16) || !aligned(layer->down, 16) || !aligned(layer->router, 16) ||
        !aligned(layer->bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(workspace, 16))
        return KQ_ERR_ALIGN;
    const int64_t n = layer->hidden;
    if ((r = kv::rows_check(x, ldx, n)) || (add && (r = kv::rows_check(add, ldadd, n))) || (r = kv::rows_check(y, ldy, n)))
        return r;
    if (y == x || (add && y == add && ldy != ldadd)) return KQ_ERR_ARG;
    const MoeSpace s = moe_space(layer, T);
    if (workspace_bytes < s.end) return KQ_ERR_SHAPE;
    if (device_check()) return KQ_ERR_DEVICE;
    uint8_t *ws = (uint8_t *)workspace;
    Moe a = {};
    a.x = x;
    a.add = add;
    a.router = layer->router;
    a.bias = layer->bias;
    a.gate = (const uint8_t *)layer->gate;
    a.up = (const uint8_t *)layer->up;
    a.down = (const uint8_t *)layer->down;
    a.y = y;
    a.ids = ids ? ids : (int32_t *)(ws + s.ids);
    a.weights = weights ? weights : (float *)(ws + s.weights);
    a.logits = (double *)ws;
    a.inner = (float *)(ws + s.inner);
    a.ldx = ldx;
    a.ldadd = ldadd;
    a.ldy = ldy;
    a.gate_bytes = gate_bytes;
    a.down_bytes = down_bytes;
    a.scale = layer->scale;
    a.E = layer->E;
    a.k = layer->k;
    a.hidden = (int)layer->hidden;
    a.n_inner = (int)layer->inner;
    a.T = T;
    a.score = layer->score;
    a.renorm = layer->renorm;
    a.act = layer->act;
    hipStream_t st = (hipStream_t)stream;
    launch_router(a, st);
    if ((r = kv::launched())) return r;
    if ((r = with_type(layer->gate_type, [&](auto tag) { return launch_gate_up<decltype(tag)::value>(a, st); }))) return r;
    return with_type(layer->down_type, [&](auto tag) { return launch_down<decltype(tag)::value>(a, st); });
}

} // extern "C"
