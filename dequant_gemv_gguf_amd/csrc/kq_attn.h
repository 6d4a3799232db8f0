// kq_attn.h -- attention of a few new tokens per request over the paged cache
// (kqkv_attn in include/kqkv.h), on the matrix cores.
//
// The mathematics.  For the rows r (a query head of one new token) that share a
// kv head, with scores s_ri = scale * q_r . k_i in units of ln 2,
//   o_r = sum_i 2^(s_ri - m_r) v_i / sum_i 2^(s_ri - m_r)
// for any m_r: the keys are cut into tiles of 32, each wave keeps a running m,
// sum l and accumulator o of its tiles, and two such states join as
//   m = max(m', m''), l = l' 2^(m' - m) + l'' 2^(m'' - m), o likewise.
// m follows the running maximum only when a score exceeds it by 2^8 (weights
// stay below 2^14 with the offset below): then o and l are rescaled; most tiles
// need neither the maximum over the lanes of a row nor a rescaling.
//
// What bounds it: every cached byte of the context is read once, for 4 * rows
// multiply-adds per fp16 key element pair at most -- HBM, as long as the loads
// stay in flight.
//
// Registers only, no staging in LDS.  Both products use the 16x16x32 matrix
// instruction, whose operands each hold 8 consecutive k per lane (row or column
// lane % 16, k = 8 (lane / 16) ..) and whose result lane holds column lane % 16,
// rows 4 (lane / 16) + i:
//   S^T = K Q^T   A = 16 keys, B = 16 rows: lane (r, g) gets 4 keys of row r
//   O^T = V^T P^T A = 16 dims, B = 16 rows: wants 8 keys of row r in lane (r, g)
// With the A rows of the two key subtiles t of a tile taken as keys
// 8 (m / 4) + 4 t + m % 4, the two results of a lane are exactly its keys
// 8 g .. 8 g + 7, so the weights go from one product to the other inside the
// lane; with V kept transposed in groups of 16 tokens its operand is one 16-byte
// load.  A lane belongs to one row throughout: m, l and masks are per lane.
//
// Precision.  A row's q is scaled by a power of two that brings its largest
// element to [2^10, 2^11) and enters as two fp16 limbs (22 bits); cached values
// enter as they are (int8 quants are whole fp16 numbers, a block's scale is
// applied to its 32-element partial score in fp32).  Weights: fp16 cache, two
// fp16 limbs of 2^6 times the weight; Q8_0 cache, the weight times the value's
// scale as three bf16 limbs (any magnitude of a scale fits).
#pragma once

#include "kq_kv.h"

namespace kq {
namespace kv {

constexpr int TILE = 32;                       // keys
constexpr int ATTN_THREADS = 256, ATTN_WAVES = 4;
constexpr float NONE = -1e30f;                 // m before the first key
constexpr float SLACK = 8.f, LIFT = 6.f;       // weights reach 2^(SLACK + LIFT) < 65504

struct Attn {
    const int32_t *ctx_len, *seq_start, *table;
    const float *q;
    float *out, *part;         // part: [item][kv head][row][dim], then [item][kv head][row] (m, l)
    int32_t *err;
    int64_t stride, ldq, ldo;
    int B, T, max_q, group, window;
    int rows_cap;              // group * max_q
    int items;                 // most pieces that all requests are cut into, >= B
    int min_tiles;             // no piece smaller than this
    int row_tiles;             // 16-row tiles per work-group: 1, 2 or 4
    float scale;               // in units of log2
};

// Tokens that a table row has room for (keys stay below 2^31 - 64, so that a
// tile's end is an int).
__device__ __forceinline__ int attn_room(const Cache &c, const Attn &a) {
    return (int)min(a.stride * (int64_t)c.page_tokens, (int64_t)INT32_MAX - 63);
}

// One request's share of the step: its rows, and the tiles [lo, lo + tiles) its
// rows see anything of.
struct Req1 {
    int first, n, ctx, tiles, lo;
};
__device__ __forceinline__ Req1 attn_req(const Cache &c, const Attn &a, int b) {
    Req1 r = {0, 0, 0, 0, 0};
    if (b >= a.B) return r;
    r.first = a.seq_start[b];
    r.n = a.seq_start[b + 1] - r.first;
    r.ctx = max(a.ctx_len[b], 0);
    if (r.n <= 0) {
        r.n = 0;
        return r;
    }
    const int hi = min(r.ctx, attn_room(c, a));
    const int64_t lo = a.window ? (int64_t)r.ctx - r.n - a.window + 1 : 0;
    r.lo = (int)(max(min(lo, (int64_t)hi), (int64_t)0) / TILE);
    r.tiles = (hi + TILE - 1) / TILE - r.lo;
    if (r.tiles < 0) r.tiles = 0;
    return r;
}

// How the requests are cut: `chunk` tiles a piece, so that there are at most
// a.items pieces (sum of max(1, ceil(tiles / chunk)) <= B + total / chunk).
__device__ __forceinline__ int attn_chunk(const Cache &c, const Attn &a, int lane) {
    if (a.items <= a.B) return INT32_MAX;
    int64_t total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) total += attn_req(c, a, b0 + lane).tiles;
#pragma unroll
    for (int s = 32; s; s >>= 1) total += __shfl_xor(total, s);
    const int64_t extra = a.items - a.B;
    return (int)max((total + extra - 1) / extra, (int64_t)a.min_tiles);
}
__device__ __forceinline__ int attn_pieces(const Req1 &r, int chunk) {
    if (r.n == 0) return 0;
    return chunk == INT32_MAX || r.tiles <= chunk ? 1 : (r.tiles + chunk - 1) / chunk;
}

// Piece `item` (b -1 when there are fewer).  All results are uniform.
struct Piece {
    int b, index, of;          // request, which of its pieces
    Req1 r;
};
__device__ __forceinline__ Piece attn_piece(const Cache &c, const Attn &a, int chunk, int item, int lane) {
    int before = 0, found = -1, index = 0, of = 0, first = 0, rn = 0, ctx = 0, tiles = 0, lo = 0;
    for (int b0 = 0; b0 < a.B && found < 0; b0 += 64) {
        const Req1 r = attn_req(c, a, b0 + lane);
        const int n = attn_pieces(r, chunk);
        int s = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d) s += o;
        }
        const int at = item - before - (s - n);
        const uint64_t hit = __ballot(at >= 0 && at < n);
        const int l = hit ? __builtin_ctzll(hit) : 0;
        if (hit) found = b0 + l;
        index = __builtin_amdgcn_readlane(at, l);
        of = __builtin_amdgcn_readlane(n, l);
        first = __builtin_amdgcn_readlane(r.first, l);
        rn = __builtin_amdgcn_readlane(r.n, l);
        ctx = __builtin_amdgcn_readlane(r.ctx, l);
        tiles = __builtin_amdgcn_readlane(r.tiles, l);
        lo = __builtin_amdgcn_readlane(r.lo, l);
        before += __builtin_amdgcn_readlane(s, 63);
    }
    return Piece{found, index, of, Req1{first, rn, ctx, tiles, lo}};
}

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef u32 u2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f4 mma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f4 mma(b8 a, b8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// 8 int8 as fp16: 0x6400 + u is 1024 + u for a byte u.
__device__ __forceinline__ h8 quants_h8(u2 x) {
    u4 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const u32 u = x[i] ^ 0x80808080u;
        w[2 * i] = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
        w[2 * i + 1] = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
    }
    h8 h = __builtin_bit_cast(h8, w);
    return h - (_Float16)1152;
}
// 8 int8 as bf16: the upper halves of their fp32 forms (7 bits at most).
__device__ __forceinline__ b8 quants_b8(u2 x) {
    u4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int v = (int)(x[i / 2] >> (16 * (i % 2)));
        const float lo = (float)(int8_t)v, hi = (float)(int8_t)(v >> 8);
        w[i] = __builtin_amdgcn_perm(__builtin_bit_cast(u32, hi), __builtin_bit_cast(u32, lo), 0x07060302u);
    }
    return __builtin_bit_cast(b8, w);
}
// x = hi + lo to 22 bits: hi rounded to zero, lo the rest.
__device__ __forceinline__ void limbs(const float *x, h8 *hi, h8 *lo) {
    u4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto h = __builtin_amdgcn_cvt_pkrtz(x[2 * i], x[2 * i + 1]);
        const auto l = __builtin_amdgcn_cvt_pkrtz(x[2 * i] - (float)h[0], x[2 * i + 1] - (float)h[1]);
        a[i] = __builtin_bit_cast(u32, h);
        b[i] = __builtin_bit_cast(u32, l);
    }
    *hi = __builtin_bit_cast(h8, a);
    *lo = __builtin_bit_cast(h8, b);
}
// x = l[0] + l[1] + l[2] to 24 bits, each limb the upper half of the rest.
__device__ __forceinline__ void limbs3(const float *x, b8 *l) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        u4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32 a = __builtin_bit_cast(u32, r[2 * i]), b = __builtin_bit_cast(u32, r[2 * i + 1]);
            w[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
            if (k < 2) {
                r[2 * i] -= __builtin_bit_cast(float, a & 0xFFFF0000u);
                r[2 * i + 1] -= __builtin_bit_cast(float, b & 0xFFFF0000u);
            }
        }
        l[k] = __builtin_bit_cast(b8, w);
    }
}

// One tile of a lane as loaded.  NB = dim / 32.
template <bool Q8, int NB> struct KTile;
template <int NB> struct KTile<false, NB> { u4 x[2][NB]; };
template <int NB> struct KTile<true, NB> { u2 x[2][NB]; h8 s[NB]; };
template <bool Q8, int NB> struct VTile;
template <int NB> struct VTile<false, NB> { u4 x[2 * NB]; };
template <int NB> struct VTile<true, NB> { u2 x[2 * NB]; h8 s[NB]; };

// lane (m, g): K rows 8 (m / 4) + 4 t + m % 4 of the tile, elements 32 s + 8 g ..;
// `at` is the 16-token group of the lane's rows.
template <bool Q8, int NB>
__device__ __forceinline__ void load_k(KTile<Q8, NB> &k, const uint8_t *mine, const uint8_t *scales, int lane) {
    constexpr int D = 32 * NB;
    const int m = lane & 15, g = lane >> 4, row = (8 * (m >> 2) + (m & 3)) & 15;
    constexpr int E = Q8 ? 1 : 2;
    const uint8_t *p = mine + row * D * E + g * 8 * E;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int s = 0; s < NB; ++s) {
            if constexpr (Q8) k.x[t][s] = *(const u2 *)(p + (4 * t * D + 32 * s));
            else k.x[t][s] = *(const u4 *)(p + (4 * t * D + 32 * s) * 2);
        }
    if constexpr (Q8) {
        const uint8_t *q = scales + (g & 1) * 16;
#pragma unroll
        for (int s = 0; s < NB; ++s) k.s[s] = *(const h8 *)(q + s * 32);
    }
}
// lane (m, g): dims 16 n + m, keys 8 g .. 8 g + 7.
template <bool Q8, int NB>
__device__ __forceinline__ void load_v(VTile<Q8, NB> &v, const uint8_t *mine, const uint8_t *scales, int lane) {
    const int m = lane & 15, g = lane >> 4;
    constexpr int E = Q8 ? 1 : 2;
    const uint8_t *p = mine + (m * 16 + (g & 1) * 8) * E;
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) {
        if constexpr (Q8) v.x[n] = *(const u2 *)(p + n * 256);
        else v.x[n] = *(const u4 *)(p + n * 512);
    }
    if constexpr (Q8) {
        const uint8_t *q = scales + (g & 1) * 16;
#pragma unroll
        for (int s = 0; s < NB; ++s) v.s[s] = *(const h8 *)(q + s * 32);
    }
}

__device__ __forceinline__ float across_groups_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float across_groups_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// One work-group: a piece of a request's tiles for one kv head and up to
// 16 * row_tiles of its rows.  Wave w takes row tile w % row_tiles and the tiles
// w / row_tiles + i * (4 / row_tiles) of the piece (waves that share a key tile
// read it through the caches); the waves of a row tile join through LDS.
template <bool Q8, int NB>
__global__ __launch_bounds__(ATTN_THREADS, NB <= 4 ? 2 : 1) void attn_kernel(Cache c, Attn a) {
    constexpr int D = 32 * NB, LD = D + 4;
    __shared__ float lds[ATTN_WAVES * 16 * (LD + 2)];   // [wave][16][LD], then [wave][16] (m, l)
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (a.rows_cap + 16 * a.row_tiles - 1) / (16 * a.row_tiles);
    // pieces that read the same keys (row groups) lie 8 blocks apart: one L2
    const int per = 8 * groups, oct = blockIdx.x / per, in = blockIdx.x - oct * per;
    const int unit = oct * 8 + (in & 7), rgroup = in >> 3;
    if (unit >= a.items * c.kv_heads) return;
    const int item = unit / c.kv_heads, head = unit - item * c.kv_heads;
    const int chunk = attn_chunk(c, a, lane);
    const Piece pc = attn_piece(c, a, chunk, item, lane);
    if (pc.b < 0) return;
    const int rows = min(pc.r.n, a.max_q) * a.group;
    const int row0 = rgroup * 16 * a.row_tiles;
    if (row0 >= rows) return;

    const int rt = wave % a.row_tiles, kw = wave / a.row_tiles, kws = ATTN_WAVES / a.row_tiles;
    const int m = lane & 15, g = lane >> 4;
    const int r = row0 + 16 * rt + m, j = r / a.group, qh = head * a.group + (r - j * a.group);
    const int64_t trow = (int64_t)pc.r.first + j;
    const bool live = r < rows && trow >= 0 && trow < a.T;
    // the row sees keys [lo, hi); hi_all and lo_all: keys that any row sees,
    // hi_min and lo_max: that every row sees
    const int64_t room = attn_room(c, a);
    const int64_t pos0 = (int64_t)pc.r.ctx - pc.r.n;
    const int hi_all = (int)min((int64_t)pc.r.ctx, room);
    const int hi_min = (int)max(min(pos0 + 1, room), (int64_t)0);
    const int lo_all = a.window ? (int)max(pos0 - a.window + 1, (int64_t)0) : 0;
    const int lo_max = a.window ? (int)max((int64_t)pc.r.ctx - a.window, (int64_t)0) : 0;
    const int hi = (int)max(min(pos0 + j + 1, room), (int64_t)0);
    const int lo = a.window ? (int)max(pos0 + j - a.window + 1, (int64_t)0) : 0;
    if ((int64_t)pc.r.ctx > room && a.err && threadIdx.x == 0) a.err[0] = 1;

    const int t0 = pc.r.lo + pc.index * (pc.of == 1 ? 0 : chunk);
    const int t1 = pc.of == 1 ? pc.r.lo + pc.r.tiles : min(t0 + chunk, pc.r.lo + pc.r.tiles);
    const int first = t0 + kw, N = first < t1 ? (t1 - first + kws - 1) / kws : 0;

    // q as two fp16 limbs
    h8 qh_[NB], ql_[NB];
    float unscale;
    {
        float x[NB][8], top = 0.f;
        const float *qp = a.q + (live ? trow : 0) * a.ldq + (int64_t)qh * D + 8 * g;
#pragma unroll
        for (int s = 0; s < NB; ++s)
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                f4 v = {0.f, 0.f, 0.f, 0.f};
                if (live) v = *(const f4 *)(qp + 32 * s + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[s][e + i] = v[i] * a.scale;
                    top = fmaxf(top, fabsf(x[s][e + i]));
                }
            }
        top = across_groups_max(top);
        int ex = 0;
        if (top > 0.f && top < INFINITY) ex = min(11 - ilogbf(top) - 1, 120);
        unscale = ldexpf(1.f, -ex);
#pragma unroll
        for (int s = 0; s < NB; ++s) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[s][e] = ldexpf(x[s][e], ex);
            limbs(x[s], &qh_[s], &ql_[s]);
        }
    }

    f4 o[2 * NB];
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) o[n] = f4{0.f, 0.f, 0.f, 0.f};
    float mx = NONE, l = 0.f;

    const u32 gp = c.page_tokens >> 4, quants = c.page_tokens * D;
    const uint8_t *kb = c.k + (u64)head * c.head_bytes, *vb = c.v + (u64)head * c.head_bytes;
    // pages of the wave's next 32 tiles: lane i holds group i % 2 of tile i / 2, page << 4 | group in page
    u32 ids = 0;
    uint64_t bad = 0;
    auto fetch_ids = [&](int n) {
        const int grp = 2 * (first + kws * (n + (lane >> 1))) + (lane & 1);
        const bool in = n + (lane >> 1) < N && grp * 16 < hi_all && grp * 16 + 16 > lo_all;
        u32 id = 0;
        bool wrong = false;
        if (in) {
            const u32 page = (u32)grp / gp;
            id = (u32)a.table[pc.b * a.stride + page];
            wrong = id >= c.n_pages;
            id = wrong ? 0 : (id << 4 | ((u32)grp - page * gp));
        }
        ids = id;
        bad = __ballot(wrong);
        if (wrong && a.err) a.err[0] = 1;
    };
    // byte offsets of the tile's two 16-token groups in K and V alike: quants or halves, and scales
    struct Where { u64 x0, x1, s0, s1; };
    auto where = [&](int n) {
        Where w;
        const u32 i0 = (u32)__builtin_amdgcn_readlane((int)ids, 2 * (n & 31));
        const u32 i1 = (u32)__builtin_amdgcn_readlane((int)ids, 2 * (n & 31) + 1);
        const u64 p0 = (u64)(i0 >> 4) * (u64)c.page_bytes, p1 = (u64)(i1 >> 4) * (u64)c.page_bytes;
        w.x0 = p0 + (i0 & 15) * (16 * D * (Q8 ? 1 : 2));
        w.x1 = p1 + (i1 & 15) * (16 * D * (Q8 ? 1 : 2));
        w.s0 = p0 + quants + (i0 & 15) * (NB * 32);
        w.s1 = p1 + quants + (i1 & 15) * (NB * 32);
        return w;
    };
    KTile<Q8, NB> kt;
    VTile<Q8, NB> vt;
    // K rows of lane m are in group m / 8, its scales and V keys in group g / 2
    auto get_k = [&](const Where &w) { load_k<Q8, NB>(kt, kb + ((m & 8) ? w.x1 : w.x0), kb + ((g & 2) ? w.s1 : w.s0), lane); };
    auto get_v = [&](const Where &w) { load_v<Q8, NB>(vt, vb + ((g & 2) ? w.x1 : w.x0), vb + ((g & 2) ? w.s1 : w.s0), lane); };

    if (N > 0) {
        fetch_ids(0);
        const Where w = where(0);
        get_k(w);
        get_v(w);
    }
    for (int n = 0; n < N; ++n) {
        // scores of the lane's 8 keys, times 1 / unscale
        float s[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            f4 d = {0.f, 0.f, 0.f, 0.f}, d2 = d;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if constexpr (Q8) {
                    const h8 k = quants_h8(kt.x[t][b]);
                    const f4 z = {0.f, 0.f, 0.f, 0.f};
                    const f4 x = mma(k, qh_[b], mma(k, ql_[b], z));
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = fmaf(x[i], (float)kt.s[b][4 * t + i], d[i]);
                } else {
                    const h8 k = __builtin_bit_cast(h8, kt.x[t][b]);
                    d = mma(k, qh_[b], d);
                    d2 = mma(k, ql_[b], d2);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * t + i] = Q8 ? d[i] : d[i] + d2[i];
        }
        const uint64_t wrong = (bad >> (2 * (n & 31))) & 3;
        const int tile = first + kws * n;
        // the next tile's keys (the last tile's again behind it)
        Where next;
        {
            const int nn = n + 1 < N ? n + 1 : n;
            if (nn != n && (nn & 31) == 0) fetch_ids(nn);
            next = where(nn);
            get_k(next);
        }
        const bool edge = wrong || tile * TILE < lo_max || tile * TILE + TILE > hi_min;
        uint32_t gone = 0;                       // keys of the lane that no row may touch
        if (edge) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int key = tile * TILE + 8 * g + e;
                const bool out = key >= hi_all || key < lo_all || ((wrong >> (g >> 1)) & 1);
                gone |= (u32)out << e;
                s[e] = out || key >= hi || key < lo ? -INFINITY : s[e];
            }
        }
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
        top *= unscale;
        if (__any(top > mx + SLACK)) {
            const float now = fmaxf(mx, across_groups_max(top));
            const float keep = __builtin_amdgcn_exp2f(mx - now);
            mx = now;
            l *= keep;
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k) o[k] *= keep;
        }
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(fmaf(s[e], unscale, LIFT - mx));
            l += p[e];
        }
        if constexpr (Q8) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = p[e] * (float)vt.s[b][e];
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = (gone >> e) & 1 ? 0.f : x[e];
                }
                b8 w[3];
                limbs3(x, w);
                const b8 v0 = quants_b8(vt.x[2 * b]), v1 = quants_b8(vt.x[2 * b + 1]);
#pragma unroll
                for (int k = 2; k >= 0; --k) {
                    o[2 * b] = mma(v0, w[k], o[2 * b]);
                    o[2 * b + 1] = mma(v1, w[k], o[2 * b + 1]);
                }
            }
        } else {
            if (edge) {
                u4 keep;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    keep[i] = ((gone >> (2 * i)) & 1 ? 0u : 0xFFFFu) | ((gone >> (2 * i + 1)) & 1 ? 0u : 0xFFFF0000u);
#pragma unroll
                for (int k = 0; k < 2 * NB; ++k) vt.x[k] &= keep;
            }
            h8 ph, pl;
            limbs(p, &ph, &pl);
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k) o[k] = mma(__builtin_bit_cast(h8, vt.x[k]), ph, o[k]);
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k) o[k] = mma(__builtin_bit_cast(h8, vt.x[k]), pl, o[k]);
        }
        get_v(next);
    }
    l = across_groups_sum(l);

    // join the waves of each row tile
    float *stat = lds + ATTN_WAVES * 16 * LD;
#pragma unroll
    for (int k = 0; k < 2 * NB; ++k) *(f4 *)(lds + (wave * 16 + m) * LD + 16 * k + 4 * g) = o[k];
    if (g == 0) {
        stat[(wave * 16 + m) * 2] = mx;
        stat[(wave * 16 + m) * 2 + 1] = l;
    }
    __syncthreads();
    const int todo = min(16 * a.row_tiles, rows - row0) * (D / 4);
    for (int i = threadIdx.x; i < todo; i += ATTN_THREADS) {
        const int rr = i / (D / 4), d = (i - rr * (D / 4)) * 4;
        float M = NONE, L = 0.f;
        f4 x = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < kws; ++w) M = fmaxf(M, stat[((w * a.row_tiles + (rr >> 4)) * 16 + (rr & 15)) * 2]);
        for (int w = 0; w < kws; ++w) {
            const int at = (w * a.row_tiles + (rr >> 4)) * 16 + (rr & 15);
            const float f = __builtin_amdgcn_exp2f(stat[at * 2] - M);
            L = fmaf(f, stat[at * 2 + 1], L);
            x += f * *(const f4 *)(lds + at * LD + d);
        }
        const int row = row0 + rr;
        if (pc.of == 1) {
            const int jj = row / a.group;
            const int64_t to = (int64_t)pc.r.first + jj;
            if (to >= 0 && to < a.T)
                *(f4 *)(a.out + to * a.ldo + (int64_t)(head * a.group + row - jj * a.group) * D + d) =
                    L == 0.f ? f4{0.f, 0.f, 0.f, 0.f} : x * (1.f / L);
        } else {
            const int64_t at = ((int64_t)item * c.kv_heads + head) * a.rows_cap + row;
            *(f4 *)(a.part + at * D + d) = x;
            if (d == 0) {
                float *ml = a.part + (int64_t)a.items * c.kv_heads * a.rows_cap * D + at * 2;
                ml[0] = M;
                ml[1] = L;
            }
        }
    }
}

// Joins the pieces of the requests that were cut: one work-group per row,
// thread (i, d) the pieces i, i + ways, ... of 4 elements.
template <int NB>
__global__ __launch_bounds__(ATTN_THREADS) void attn_join_kernel(Cache c, Attn a) {
    constexpr int D = 32 * NB, LANES = D / 4, WAYS = ATTN_THREADS / LANES;
    __shared__ f4 xs[ATTN_THREADS];
    __shared__ float ls[WAYS];
    const int lane = threadIdx.x & 63;
    const int b = blockIdx.x / (c.kv_heads * a.rows_cap), left = blockIdx.x - b * (c.kv_heads * a.rows_cap);
    const int head = left / a.rows_cap, row = left - head * a.rows_cap;
    const int chunk = attn_chunk(c, a, lane);
    // the request's first piece: the pieces before it
    int before = 0;
    Req1 mine = {0, 0, 0, 0, 0};
    for (int b0 = 0; b0 <= b; b0 += 64) {
        const Req1 r = attn_req(c, a, b0 + lane);
        int n = b0 + lane < b ? attn_pieces(r, chunk) : 0;
#pragma unroll
        for (int s = 32; s; s >>= 1) n += __shfl_xor(n, s);
        before += n;
        if (b < b0 + 64) {
            mine.first = __builtin_amdgcn_readlane(r.first, b - b0);
            mine.n = __builtin_amdgcn_readlane(r.n, b - b0);
            mine.tiles = __builtin_amdgcn_readlane(r.tiles, b - b0);
        }
    }
    const int pieces = attn_pieces(mine, chunk);
    if (pieces <= 1 || row >= min(mine.n, a.max_q) * a.group) return;
    const float *ml = a.part + (int64_t)a.items * c.kv_heads * a.rows_cap * D;
    auto at = [&](int i) { return ((int64_t)(before + i) * c.kv_heads + head) * a.rows_cap + row; };
    float M = NONE;
    for (int i = lane; i < pieces; i += 64) M = fmaxf(M, ml[at(i) * 2]);
#pragma unroll
    for (int s = 32; s; s >>= 1) M = fmaxf(M, __shfl_xor(M, s));
    const int way = threadIdx.x / LANES, d = (threadIdx.x - way * LANES) * 4;
    f4 x = {0.f, 0.f, 0.f, 0.f};
    float L = 0.f;
    if (way < WAYS) {
        for (int i = way; i < pieces; i += WAYS) {
            const int64_t k = at(i);
            const float f = __builtin_amdgcn_exp2f(ml[k * 2] - M);
            L = fmaf(f, ml[k * 2 + 1], L);
            x += f * *(const f4 *)(a.part + k * D + d);
        }
        if (d == 0) ls[way] = L;
    }
    xs[threadIdx.x] = x;
    __syncthreads();
    if (way == 0) {
        for (int w = 1; w < WAYS; ++w) {
            x += xs[w * LANES + threadIdx.x];
            L += ls[w];
        }
        const int j = row / a.group;
        const int64_t to = (int64_t)mine.first + j;
        if (to >= 0 && to < a.T)
            *(f4 *)(a.out + to * a.ldo + (int64_t)(head * a.group + row - j * a.group) * D + d) =
                L == 0.f ? f4{0.f, 0.f, 0.f, 0.f} : x * (1.f / L);
    }
}

template <int NB> int launch_attn(bool q8, const Cache &c, const Attn &a, hipStream_t st);

} // namespace kv
} // namespace kq
