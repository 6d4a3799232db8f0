// kq_kv.h -- what the paged-cache translation units share: the cache as the
// kernels see it, its address arithmetic and its argument checks.  C ABI and
// layout in include/kqkv.h.
#pragma once

#include "kq_impl.h"
#include "kqkv.h"

namespace kq {

// Whether the current device is a gfx950 (kqgemv.hip).
__attribute__((visibility("hidden"))) int device_check();

namespace kv {

typedef uint64_t u64;
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));

// The cache in a kernel's arguments.  Offsets inside one head of a page stay
// below 2^18 bytes; a page's offset is 64-bit.
struct Cache {
    uint8_t *k, *v;
    int64_t page_bytes;
    u32 head_bytes;        // of one head of a page
    u32 page_tokens;       // P
    u32 slots;             // n_pages * P
    u32 n_pages;
    int kv_heads, dim;
};

template <bool Q8> struct Elem;
template <> struct Elem<false> { typedef _Float16 type; };
template <> struct Elem<true> { typedef int8_t type; };

// Index of element (token t, element d) of one head of a page, in K and in V,
// and of a Q8_0 scale after the P * D quants.
__device__ __forceinline__ u32 k_at(u32 t, u32 d, u32 dim) { return t * dim + d; }
__device__ __forceinline__ u32 v_at(u32 t, u32 d, u32 dim) { return (t >> 4) * 16 * dim + d * 16 + (t & 15); }
__device__ __forceinline__ u32 scale_at(u32 t, u32 b, u32 dim) {
    return (t >> 4) * (dim >> 5) * 16 + b * 16 + (t & 15);
}

// The scale and the quants' divisor of a block whose largest magnitude has the
// bits m (magnitudes order like integers, NaN on top).  The 127th is a product
// with the reciprocal: beside the rounding to fp16 the difference to a quotient
// is nothing (2^-23 of it), but it decides about one block in 10^6 that lies
// between two fp16 scales, so it is part of the format.
struct Scale {
    float s;               // fp16, as stored
    bool none;             // every quant is 0
};
__device__ __forceinline__ Scale block_scale(u32 m) {
    const bool bad = m >= 0x7F800000u;
    const float s = (float)(_Float16)fminf(__builtin_bit_cast(float, m) * (1.f / 127.f), 65504.f);
    return Scale{bad ? __builtin_nanf("") : s, bad || s == 0.f};
}
__device__ __forceinline__ int quant(float x, const Scale &s) {
    return s.none ? 0 : (int)fmaxf(-127.f, fminf(127.f, rintf(x / s.s)));
}
__device__ __forceinline__ u32 magnitude(float x) { return __builtin_bit_cast(u32, x) & 0x7FFFFFFFu; }
__device__ __forceinline__ u32 magnitude(f4 x) {
    return max(max(magnitude(x[0]), magnitude(x[1])), max(magnitude(x[2]), magnitude(x[3])));
}

inline int cache_limits(int type, int kv_heads, int head_dim, int page_tokens) {
    if (type != KQKV_F16 && type != KQKV_Q8_0) return KQ_ERR_TYPE;
    if (kv_heads < 1 || kv_heads > 1024) return KQ_ERR_SHAPE;
    if (head_dim < 32 || head_dim > 256 || head_dim % 32) return KQ_ERR_SHAPE;
    if (page_tokens < 16 || page_tokens > 256 || page_tokens % 16) return KQ_ERR_SHAPE;
    return KQ_OK;
}

// Every check of a cache argument that any call makes.
inline int cache_check(const kqkv_cache *c) {
    if (!c) return KQ_ERR_NULL;
    const int r = cache_limits(c->type, c->kv_heads, c->head_dim, c->page_tokens);
    if (r) return r;
    if (c->n_pages < 1 || c->n_pages > (INT32_MAX / c->page_tokens)) return KQ_ERR_SHAPE;
    if (!c->k || !c->v) return KQ_ERR_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return KQ_ERR_ALIGN;
    return KQ_OK;
}

inline Cache cache_args(const kqkv_cache *c) {
    Cache a;
    a.k = (uint8_t *)c->k;
    a.v = (uint8_t *)c->v;
    const u32 n = (u32)(c->page_tokens * c->head_dim);
    a.head_bytes = c->type == KQKV_F16 ? 2 * n : n + n / 16;
    a.page_bytes = (int64_t)a.head_bytes * c->kv_heads;
    a.page_tokens = (u32)c->page_tokens;
    a.slots = (u32)(c->n_pages * c->page_tokens);
    a.n_pages = (u32)c->n_pages;
    a.kv_heads = c->kv_heads;
    a.dim = c->head_dim;
    return a;
}

// fp32 rows: a pointer, its row stride and the row length.
inline int rows_check(const void *p, int64_t ld, int64_t n) {
    if (!p) return KQ_ERR_NULL;
    if (!aligned(p, 16) || ld % 4) return KQ_ERR_ALIGN;
    if (ld < n || ld > ((int64_t)1 << 40)) return KQ_ERR_SHAPE;
    return KQ_OK;
}

inline int launched() { return hipGetLastError() == hipSuccess ? KQ_OK : KQ_ERR_LAUNCH; }

} // namespace kv
} // namespace kq
