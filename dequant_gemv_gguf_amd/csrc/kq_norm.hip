// kq_norm.hip -- the residual's addition and the root-mean-square norm of
// include/kqstep.h.
//
// Bound: HBM (x and add read, sum and y written, once): 8192 rows of 8192 with both
// take 193 us, 5.6 TB/s; for few rows the chain of one row, a load, the sum of its
// squares, a store: one row of 2048 takes 2.6 us, 250 x 32 heads of 128 3.3.  A row (a
// token's, or one of its heads) stays in registers from the load to the stores.  Rows
// of up to 512 elements take 16, 32 or 64 lanes, so that a wave holds up to four heads;
// longer ones a work-group.  The sum of squares and y are computed in 64 bits: at one
// square and two products an element that costs nothing beside the loads, and y is the
// correctly rounded result for all but ties of 2^-29.  Q8_0 rows: 4099 of 4096 with
// fp32 rows, sum and add take 58 us (5.0 TB/s), 49 without them (5.5 TB/s).
#include "kq_step.h"

#include <cmath>

namespace kq {
namespace step {

using kv::Scale;
using kv::block_scale;
using kv::magnitude;
using kv::quant;

constexpr int NORM_THREADS = 256;

struct Norm {
    const float *x, *add, *weight;
    float *sum, *y;
    uint8_t *y8;
    int64_t ldx, ldadd, ldsum, ldy, row8;
    double eps, inv_n;
    int heads, n;
    u32 rows;               // T * heads
    u32 first;              // the launch's first row (a grid holds fewer than 2^32 threads)
};

// Where one row is.
struct NormRow {
    const float *x, *add;
    float *sum, *y;
    uint8_t *y8;
};
__device__ __forceinline__ NormRow norm_row(const Norm &a, u32 row) {
    const u32 t = row / (u32)a.heads, h = row - t * (u32)a.heads;
    const int64_t o = (int64_t)h * a.n;
    return NormRow{a.x + t * a.ldx + o, a.add ? a.add + t * a.ldadd + o : nullptr, a.sum ? a.sum + t * a.ldsum + o : nullptr,
                   a.y ? a.y + t * a.ldy + o : nullptr, a.y8 ? a.y8 + t * a.row8 + (int64_t)h * (a.n / 32) * 34 : nullptr};
}

__device__ __forceinline__ double squares(f4 h) {
    const double a = h[0], b = h[1], c = h[2], d = h[3];
    return (a * a + b * b) + (c * c + d * d);
}

__device__ __forceinline__ f4 normed(f4 h, const float *weight, int e, double r) {
    const f4 w = weight ? *(const f4 *)(weight + e) : f4{1.f, 1.f, 1.f, 1.f};
    f4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (float)((double)h[i] * (double)w[i] * r);
    return y;
}

// y's elements e .. e + 3 of a row into its Q8_0 blocks: the 8 lanes of a block
// find its scale (every lane of the block is here: n is a multiple of 32).
__device__ __forceinline__ void store8(uint8_t *row, int e, f4 y) {
    u32 m = magnitude(y);
    m = max(m, (u32)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
    m = max(m, (u32)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
    m = max(m, (u32)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
    const Scale s = block_scale(m);
    uint8_t *b = row + (e >> 5) * 34;
    if ((e & 31) == 0) *(_Float16 *)b = (_Float16)s.s;
    uint16_t *q = (uint16_t *)(b + 2 + (e & 31));
    q[0] = (uint16_t)((quant(y[0], s) & 0xFF) | (quant(y[1], s) & 0xFF) << 8);
    q[1] = (uint16_t)((quant(y[2], s) & 0xFF) | (quant(y[3], s) & 0xFF) << 8);
}

// Keeps h as it is in registers, one piece after the other: without it the compiler
// holds on to the 64-bit values of all of a lane's pieces (240 registers for 8).
__device__ __forceinline__ void pin(f4 &h) { asm volatile("" : "+v"(h)); }

// A row's pieces at 4 (i + STEP v), v < V, zeros past its end.  (Read from the
// row's start there: a branch around each load makes the compiler move the whole
// array at every one of them.)
template <int STEP, int V> __device__ __forceinline__ void load_row(const NormRow &r, int i, int n, f4 (&h)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 4 * (i + STEP * v);
        h[v] = *(const f4 *)(r.x + (e < n ? e : 0));
    }
    if (r.add) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = 4 * (i + STEP * v);
            h[v] += *(const f4 *)(r.add + (e < n ? e : 0));
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 4 * (i + STEP * v) < n ? h[v] : f4{0.f, 0.f, 0.f, 0.f};
}

// V pieces of 4 elements a lane, LANES * 4 elements apart, n <= 4 V LANES.
template <int LANES, int V>
__global__ __launch_bounds__(NORM_THREADS) void norm_lanes_kernel(const Norm a) {
    const int lane = threadIdx.x % LANES;
    const u32 row = a.first + blockIdx.x * (u32)(NORM_THREADS / LANES) + threadIdx.x / LANES;
    if (row >= a.rows) return;
    const NormRow r = norm_row(a, row);
    f4 h[V];
    load_row<LANES>(r, lane, a.n, h);
    double s = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        pin(h[v]);
        s += squares(h[v]);
    }
    s = sum_d<LANES>(s);
    const double f = 1.0 / sqrt(s * a.inv_n + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 4 * (lane + LANES * v);
        pin(h[v]);
        if (e < a.n) {
            if (r.sum) *(f4 *)(r.sum + e) = h[v];
            const f4 y = normed(h[v], a.weight, e, f);
            if (r.y) *(f4 *)(r.y + e) = y;
            if (r.y8) store8(r.y8, e, y);
        }
    }
}

// A work-group a row; V 0: rows of any length, read twice.
template <int THREADS, int V>
__global__ __launch_bounds__(THREADS) void norm_row_kernel(const Norm a) {
    __shared__ double waves[THREADS / 64];
    const NormRow r = norm_row(a, a.first + blockIdx.x);
    double s = 0.0;
    f4 h[V ? V : 1];
    if (V) {
        load_row<THREADS>(r, threadIdx.x, a.n, h);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            pin(h[v]);
            s += squares(h[v]);
        }
    } else {
        for (int e = 4 * threadIdx.x; e < a.n; e += 4 * THREADS)
            s += squares(r.add ? *(const f4 *)(r.x + e) + *(const f4 *)(r.add + e) : *(const f4 *)(r.x + e));
    }
    s = sum_d<64>(s);
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) s += waves[w];
    const double f = 1.0 / sqrt(s * a.inv_n + a.eps);
    auto out = [&](int e, f4 h) {
        if (r.sum) *(f4 *)(r.sum + e) = h;
        const f4 y = normed(h, a.weight, e, f);
        if (r.y) *(f4 *)(r.y + e) = y;
        if (r.y8) store8(r.y8, e, y);
    };
    if (V) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = 4 * ((int)threadIdx.x + THREADS * v);
            pin(h[v]);
            if (e < a.n) out(e, h[v]);
        }
    } else {
        // (a thread writes the elements that it has read, and no others)
        for (int e = 4 * threadIdx.x; e < a.n; e += 4 * THREADS)
            out(e, r.add ? *(const f4 *)(r.x + e) + *(const f4 *)(r.add + e) : *(const f4 *)(r.x + e));
    }
}

// `per` rows a work-group, at most 2^21 work-groups a launch.
template <class Kern> static void launch_rows(Kern kern, Norm a, u32 per, int threads, hipStream_t st) {
    for (;;) {
        const u32 wgs = (a.rows - a.first - 1) / per + 1, now = std::min(wgs, 1u << 21);
        hipLaunchKernelGGL(kern, dim3(now), dim3(threads), 0, st, a);
        if (now == wgs) return;
        a.first += now * per;
    }
}
template <int LANES, int V> static void launch_lanes(const Norm &a, hipStream_t st) {
    launch_rows(norm_lanes_kernel<LANES, V>, a, NORM_THREADS / LANES, NORM_THREADS, st);
}
template <int THREADS, int V> static void launch_row(const Norm &a, hipStream_t st) {
    launch_rows(norm_row_kernel<THREADS, V>, a, 1, THREADS, st);
}

} // namespace step
} // namespace kq

using namespace kq;
using namespace kq::step;

extern "C" int kqstep_norm(int T, int heads, int n, const float *x, int64_t ldx, const float *add, int64_t ldadd,
                           float *sum, int64_t ldsum, const float *weight, float eps, float *y, int64_t ldy, void *y8,
                           void *stream) {
    if (T < 0 || T >= (1 << 23) || heads < 1 || heads > 1024 || n < 4 || n % 4 || n > (1 << 20)) return KQ_ERR_SHAPE;
    const int64_t row = (int64_t)heads * n;
    if (row > (1 << 20) || (int64_t)T * heads > INT32_MAX || (y8 && n % 32)) return KQ_ERR_SHAPE;
    if (!(eps >= 0.f) || !std::isfinite(eps) || (sum && !add)) return KQ_ERR_ARG;
    if (T == 0) return KQ_OK;
    if (!y && !y8) return KQ_ERR_NULL;
    int r;
    if ((r = kv::rows_check(x, ldx, row)) || (add && (r = kv::rows_check(add, ldadd, row))) ||
        (sum && (r = kv::rows_check(sum, ldsum, row))) || (y && (r = kv::rows_check(y, ldy, row))))
        return r;
    if (!aligned(weight, 16) || !aligned(y8, 16)) return KQ_ERR_ALIGN;
    if ((sum == x && ldsum != ldx) || (add && sum == add && ldsum != ldadd) || (y == x && ldy != ldx) ||
        (add && y == add && ldy != ldadd))
        return KQ_ERR_ARG;
    if (y && y == sum) return KQ_ERR_ARG;
    if (device_check()) return KQ_ERR_DEVICE;
    const Norm a = {x, add, weight, sum, y, (uint8_t *)y8, ldx, ldadd, ldsum, ldy, row / 32 * 34, eps, 1.0 / n, heads, n,
                    (u32)(T * heads), 0};
    hipStream_t st = (hipStream_t)stream;
    // The threads of a row: fewer wait less for each other where there are many rows,
    // more have a shorter chain each.  Measured, us, one row / many rows:
    //   64 lanes with 2 of 4 idle for heads of 64, 128 (4096 x 64 and 32 heads): 75 and 43, as here 27 and 27
    //   512: a work-group of 128 threads 2.1 / 67 (65536 rows), 64 lanes 2.2 / 49
    //   1024: 64 lanes 2.6 / 48.9 (32768 rows), 128 threads 2.3 / 47.7, 256 2.0 / 48.0 (8192 rows: 11.8, 12.3, 12.9)
    //   2048: 64 lanes 3.4 / 51.6 (16384 rows), 256 threads 2.3 / 48.3, 512 2.1 / 47.9 (4096 rows: 12.5, 13.1)
    //   4096: 256 threads 3.0 / 48.7 (8192 rows), 512 2.6 / 47.9, 1024 2.7 / 57.0
    //   8192: 256 threads 4.0 / 51.9 (4096 rows), 512 3.2 / 50.9, 1024 3.2 / 50.0 (rows of 5120: 35.5, 33.9, 37.3)
    //   32768: in registers 5.6 / 57 (1024 rows), read twice 7.0 / 72
    if (n <= 64) launch_lanes<16, 1>(a, st);
    else if (n <= 128) launch_lanes<32, 1>(a, st);
    else if (n <= 256) launch_lanes<64, 1>(a, st);
    else if (n <= 512) launch_lanes<64, 2>(a, st);
    else if (n <= 1024) launch_row<128, 2>(a, st);
    else if (n <= 2048) launch_row<256, 2>(a, st);
    else if (n <= 4096) launch_row<512, 2>(a, st);
    else if (n <= 8192) launch_row<512, 4>(a, st);
    else if (n <= 16384) launch_row<1024, 4>(a, st);
    else if (n <= 32768) launch_row<1024, 8>(a, st);
    else launch_row<1024, 0>(a, st);
    return kv::launched();
}
