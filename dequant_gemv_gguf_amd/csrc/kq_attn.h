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
// What bounds it: every cached byte of the context is read once, and each pair of
// a key's and a value's element takes part in 2 multiply-adds a row (in limbs,
// 4 or 5): HBM for up to 16 rows, as long as the loads stay in flight.
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
// element to [2^10, 2^11) and enters as two fp16 limbs (22 bits), and so do the
// weights, times 2^6: rounded at 2^-25, 2^-31 of the largest weight, which takes
// bits from those below 2^-9 of it.
// fp16 keys and values enter as they are.  Int8 quants of keys are whole fp16
// numbers, a block's scale is applied to its 32-element partial score in fp32;
// an int8 value, scale times quant (19 bits, a multiple of 2^-24), is exactly the
// half it rounds to and the half that remains.  Of the products of two two-limb
// numbers the one of both low limbs is left out (2^-22).
//
// Measured (MI355X, 64 query heads, 8 kv heads, head size 128): one request of
// 131072 fp16 tokens 90 to 94 us (5.7 to 6.0 TB/s of K and V); 64 requests of up to
// 32768 Q8_0 tokens 289 us (5.4 TB/s); one of 37 tokens 5.8 us; eight rows of 4
// requests of up to 16384 Q8_0 tokens 57 us, of the kernel's 49 the vector units
// work 43 % and the matrix units 18 %; of 8 of 4096 tokens 45 us (fp16) and 44;
// eight rows of 4 of 4096, 8 query heads and one kv head of 256, 30 and 33.
#pragma once

#include "kq_kv.h"

namespace kq {
namespace kv {

constexpr int TILE = 32;                       // keys
constexpr int ATTN_THREADS = 256, ATTN_WAVES = 4;
// Waves per SIMD that the registers are cut for (a tile, o and the softmax), so that no kernel spills.
constexpr int ATTN_OCCUPANCY(int NB, int RT) { return RT == 1 ? (NB <= 4 ? 3 : NB <= 6 ? 2 : 1) : NB <= 2 ? 3 : 2; }
// Head sizes that have kernels with two row tiles a wave (past them, the registers do not suffice).
constexpr int TWO_TILES_NB = 4;
constexpr float NONE = -3e38f;                 // m before the first key
constexpr float SLACK = 8.f, LIFT = 6.f;       // weights reach 2^(SLACK + LIFT) < 65504

struct Attn {
    const int32_t *ctx_len, *seq_start, *table;
    const float *q;
    float *out, *part;         // part: [item][kv head][row] of dim outputs, m, l, 2 unused
    int4 *info;                // [request] items of its first whole piece and of its last one, pieces
    int32_t *err;
    int64_t stride, ldq, ldo;
    int B, T, max_q, group, window;
    int rows_cap;              // group * max_q
    int items;                 // most pieces that all requests are cut into, >= B
    int min_tiles;             // no piece smaller than this
    int row_waves;             // waves of a work-group that differ in their rows: 1, 2 or 4
    u32 group_magic, gp_magic; // ceil(2^32 / d) for d = group and page_tokens / 16: x / d is the upper half of x * magic
                               // while x * d < 2^32 (x < rows_cap) or, with d <= 16, x < 2^28 (a 16-token group)
    float scale;               // in units of log2
};

// Tokens that a table row has room for (keys stay below 2^31 - 64, so that a
// tile's end is an int).
__device__ __forceinline__ int attn_room(const Cache &c, const Attn &a) {
    return (int)min(a.stride * (int64_t)c.page_tokens, (int64_t)INT32_MAX - 63);
}

__device__ __forceinline__ int div_magic(int x, u32 magic) { return magic ? (int)__umulhi((u32)x, magic) : x; }

// One request's share of the step: its rows, and the tiles [lo, lo + tiles) its
// rows see anything of.
struct Req1 {
    int first, n, ctx, tiles, lo;
};
__device__ __forceinline__ Req1 attn_req(const Cache &c, const Attn &a, int b) {
    const bool in = b < a.B;
    const int i = in ? b : 0;
    const int first = a.seq_start[i], end = a.seq_start[i + 1], ctx = max(a.ctx_len[i], 0);
    Req1 r;
    r.first = first;
    r.n = in ? max(end - first, 0) : 0;
    r.ctx = ctx;
    const int hi = min(ctx, attn_room(c, a));
    const int64_t lo = a.window ? (int64_t)ctx - r.n - a.window + 1 : 0;
    r.lo = (int)(max(min(lo, (int64_t)hi), (int64_t)0) / TILE);
    r.tiles = r.n ? max((hi + TILE - 1) / TILE - r.lo, 0) : 0;
    return r;
}

// Inclusive prefix sums over the wave, in registers (row shifts, then the row
// broadcasts).
template <int CTRL, int ROWS> __device__ __forceinline__ int dpp_or_0(int x) {
    return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int x) {
    x += dpp_or_0<0x111, 0xF>(x);
    x += dpp_or_0<0x112, 0xF>(x);
    x += dpp_or_0<0x114, 0xF>(x);
    x += dpp_or_0<0x118, 0xF>(x);
    x += dpp_or_0<0x142, 0xA>(x);
    return x + dpp_or_0<0x143, 0xC>(x);
}
__device__ __forceinline__ float wave_sum(float x) {
    auto add = [](float v, int o) { return v + __builtin_bit_cast(float, o); };
    auto bits = [](float v) { return __builtin_bit_cast(int, v); };
    x = add(x, dpp_or_0<0x111, 0xF>(bits(x)));
    x = add(x, dpp_or_0<0x112, 0xF>(bits(x)));
    x = add(x, dpp_or_0<0x114, 0xF>(bits(x)));
    x = add(x, dpp_or_0<0x118, 0xF>(bits(x)));
    x = add(x, dpp_or_0<0x142, 0xA>(bits(x)));
    x = add(x, dpp_or_0<0x143, 0xC>(bits(x)));
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(bits(x), 63));
}

// How the requests are cut: whole pieces of `chunk` tiles, and a last one of at
// least chunk / 8 (and 1) and less than chunk more than that (a request's only
// one may be shorter), so that there are at most a.items pieces.  total / (items - B) is
// always enough: sum of whole ones <= total / chunk <= items - B, and a last one
// each.  (The sum of up to 4096 counts is taken in fp32 and raised by 2^-16,
// more than its rounding.)  With up to 64 requests, one a lane, smaller chunks
// from total / items on are tried, which make as many pieces as there may be
// (16 requests of 4096 Q8_0 tokens and 8 rows 87 -> 74 us, 32 of 8192 fp16
// tokens and heads of 160 295 -> 221).
// All whole pieces come before all last ones: the work-groups that start last
// are the short ones.  (r0: the lane's request of the first 64.)
__device__ __forceinline__ int whole_pieces(const Req1 &r, int chunk) {
    const int least = max(chunk / 8, 1);
    return r.tiles > least ? (int)((u32)(r.tiles - least) / (u32)chunk) : 0;
}
__device__ __forceinline__ int attn_chunk(const Cache &c, const Attn &a, const Req1 &r0, int lane) {
    if (a.items <= a.B) return INT32_MAX;
    float total = wave_sum((float)r0.tiles);
    for (int b0 = 64; b0 < a.B; b0 += 64) total += wave_sum((float)attn_req(c, a, b0 + lane).tiles);
    const float each = total * (1.f + 1.f / 65536.f) / (float)(a.items - a.B);
    int hi = max(__builtin_amdgcn_readfirstlane((int)fminf(each, 1e9f)) + 1, a.min_tiles);
    if (a.B > 64 || a.B == 1) return hi;
    int lo = max(__builtin_amdgcn_readfirstlane((int)fminf(total / (float)a.items, 1e9f)), a.min_tiles);
    for (int i = 0; i < 4 && lo < hi; ++i) {
        const int at = i ? (lo + hi) / 2 : lo;
        const int pieces = __builtin_amdgcn_readlane(wave_scan(r0.n ? whole_pieces(r0, at) + 1 : 0), 63);
        if (pieces <= a.items) hi = at;
        else lo = at + 1;
    }
    return hi;
}

// Piece `item` (b -1 when there are fewer).  All results are uniform.
struct Piece {
    int b, index, of;          // request, which of its pieces
    int whole, last;           // the items of its first whole piece and of its last one
    Req1 r;
};
__device__ __forceinline__ Piece attn_piece(const Cache &c, const Attn &a, const Req1 &r0, int chunk, int item,
                                            int lane) {
    if (a.items <= a.B) {                            // one piece a request
        const Req1 r = attn_req(c, a, item);
        return Piece{r.n ? item : -1, 0, 1, 0, item, r};
    }
    int found = -1, index = 0, of = 0, w0 = 0, last0 = 0, first = 0, rn = 0, ctx = 0, tiles = 0, lo = 0;
    int wholes = 0;
    if (a.B > 64)
        for (int b0 = 0; b0 < a.B; b0 += 64)
            wholes += __builtin_amdgcn_readlane(wave_scan(whole_pieces(attn_req(c, a, b0 + lane), chunk)), 63);
    int wbefore = 0, lbefore = 0;
    for (int b0 = 0; b0 < a.B && found < 0; b0 += 64) {
        const Req1 r = b0 ? attn_req(c, a, b0 + lane) : r0;
        const int w = whole_pieces(r, chunk), any = r.n ? 1 : 0;
        const int ws = wave_scan(w), ls = wave_scan(any);
        if (a.B <= 64) wholes = __builtin_amdgcn_readlane(ws, 63);
        const int wf = wbefore + ws - w, lf = wholes + lbefore + ls - any;
        const bool in_w = item >= wf && item < wf + w, in_l = any && item == lf;
        const uint64_t hit = __ballot(in_w || in_l);
        const int l = hit ? __builtin_ctzll(hit) : 0;
        if (hit) found = b0 + l;
        index = __builtin_amdgcn_readlane(in_l ? w : item - wf, l);
        of = __builtin_amdgcn_readlane(w + 1, l);
        w0 = __builtin_amdgcn_readlane(wf, l);
        last0 = __builtin_amdgcn_readlane(lf, l);
        first = __builtin_amdgcn_readlane(r.first, l);
        rn = __builtin_amdgcn_readlane(r.n, l);
        ctx = __builtin_amdgcn_readlane(r.ctx, l);
        tiles = __builtin_amdgcn_readlane(r.tiles, l);
        lo = __builtin_amdgcn_readlane(r.lo, l);
        wbefore += __builtin_amdgcn_readlane(ws, 63);
        lbefore += __builtin_amdgcn_readlane(ls, 63);
    }
    return Piece{found, index, of, w0, last0, Req1{first, rn, ctx, tiles, lo}};
}

typedef u32 u2 __attribute__((ext_vector_type(2)));
typedef unsigned short us8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f4 mma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// 8 int8 q as fp16: 0x6400 + u is 1024 + u for the byte u = q + 128.
__device__ __forceinline__ h8 quants_h8(u32 x0, u32 x1) {
    u4 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const u32 u = (i ? x1 : x0) ^ 0x80808080u;
        w[2 * i] = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
        w[2 * i + 1] = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
    }
    return __builtin_bit_cast(h8, w) - (_Float16)1152;
}
// (q + 128) 2^-24: the bytes as fp16 subnormals, which the matrix instructions
// take as they are; two operations less per four quants where the 128 comes
// off elsewhere.
__device__ __forceinline__ h8 biased_h8(u32 x0, u32 x1) {
    u4 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const u32 u = (i ? x1 : x0) ^ 0x80808080u;
        w[2 * i] = __builtin_amdgcn_perm(0u, u, 0x0C010C00u);
        w[2 * i + 1] = __builtin_amdgcn_perm(0u, u, 0x0C030C02u);
    }
    return __builtin_bit_cast(h8, w);
}
// x minus a half of h, exactly, in one operation (written as a difference it is
// a conversion and a subtraction).
__device__ __forceinline__ float minus_lo(u32 h, float x) {
    float r;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r) : "v"(h), "v"(x));
    return r;
}
__device__ __forceinline__ float minus_hi(u32 h, float x) {
    float r;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r) : "v"(h), "v"(x));
    return r;
}
// x = hi + lo to 22 bits: hi rounded to zero, lo the rest, rounded to nearest (where it is subnormal, at 2^-25, a rounding
// to zero would take from every small weight of a row, and nothing from their sum).
__device__ __forceinline__ void limbs(const float *x, h8 *hi, h8 *lo) {
    u4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_pkrtz(x[2 * i], x[2 * i + 1]));
        const f2 rest = {minus_lo(a[i], x[2 * i]), minus_hi(a[i], x[2 * i + 1])};
        b[i] = __builtin_bit_cast(u32, __builtin_convertvector(rest, hf2));
    }
    *hi = __builtin_bit_cast(h8, a);
    *lo = __builtin_bit_cast(h8, b);
}

// A tile's K and V of a lane as loaded (16 bytes an instruction and lane
// wherever the rows allow it).  NB = dim / 32.
template <bool Q8, int NB> struct Tile {
    static constexpr int W = Q8 ? 2 : 4;   // dwords of one operand
    u32 k[2][NB * W], v[2 * NB * W];
    h8 s;                      // Q8_0: 16 bytes of the tile's scales
    u32 wrong;                 // bit u: group u lies in a page that is none
};

// A K operand of 16 rows wants 4 pieces of every row at once, but a load that
// takes 64 bytes of 16 rows asks the cache for twice as many lines as one that
// takes 128 bytes of 8 rows, and those requests are what the stream waits for.
// So a unit of 128 bytes of a row (two fp16 operands, or four int8 ones) is
// loaded for rows 0..7 (the tile's first 16-token group) by one instruction and
// for rows 8..15 (the second) by another, lane (m, g) taking 16-byte piece
// 4 (m / 8) + g of row m % 8; half of the lanes' registers then change places
// across the row of 16 lanes.
constexpr int ROW_ROR8 = 0x128;
__device__ __forceinline__ void swap_rows(u32 &x, u32 &y) {
    const int p = __builtin_amdgcn_update_dpp((int)x, (int)y, ROW_ROR8, 0xF, 0xC, false);
    const int q = __builtin_amdgcn_update_dpp((int)y, (int)x, ROW_ROR8, 0xF, 0x3, false);
    x = (u32)p;
    y = (u32)q;
}
// Lanes 32..63 of x change places with lanes 0..31 of y; odd rows of 16 lanes
// of x with even ones of y.
__device__ __forceinline__ void swap_halves(u32 &x, u32 &y) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0];
    y = r[1];
}
__device__ __forceinline__ void swap_odd_rows(u32 &x, u32 &y) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    x = r[0];
    y = r[1];
}

// NT: the cache lines are not to be kept (whole lines are asked for, once).
template <bool NT> __device__ __forceinline__ u4 load16(const uint8_t *p) {
    return NT ? __builtin_nontemporal_load((const u4 *)p) : *(const u4 *)p;
}

// Row of K that lane m's operand stands for in subtile t, within its group:
// 8 (m / 4 % 2) + 4 t + m % 4 (keys 8 (m / 4) + 4 t + m % 4 of the tile).
// k0, k1: the head's rows of the tile's two groups.
template <bool Q8, int NB, bool NT>
__device__ __forceinline__ void load_k(Tile<Q8, NB> &to, const uint8_t *k0, const uint8_t *k1, int lane) {
    constexpr int E = Q8 ? 1 : 2, RB = 32 * NB * E, UNITS = RB / 128, W = Tile<Q8, NB>::W;
    const int m = lane & 15, g = lane >> 4, row = 8 * ((m >> 2) & 1) + (m & 3);
    const u32 at = row * RB + ((m >> 3) * 4 + g) * 16;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const u4 a = load16<NT>(k0 + at + (4 * t * RB + 128 * u)), b = load16<NT>(k1 + at + (4 * t * RB + 128 * u));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                to.k[t][8 * u + i] = a[i];
                to.k[t][8 * u + 4 + i] = b[i];
            }
        }
    // what is left of a row: 64 bytes as they are, then (int8) 32
    if constexpr (RB % 128 != 0) {
        const u64 step = (u64)(k1 - k0);
        const uint8_t *p = k0 + ((m & 8) ? step : 0) + row * RB + 128 * UNITS;
        constexpr int DONE = 8 * UNITS;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (RB % 128 >= 64) {
                const u4 a = *(const u4 *)(p + 16 * g + 4 * t * RB);
#pragma unroll
                for (int i = 0; i < 4; ++i) to.k[t][DONE + i] = a[i];
            }
            if constexpr (RB % 64 != 0) {
                const u2 a = *(const u2 *)(p + (RB % 128 - 32) + 16 * (g & 1) + 8 * (g >> 1) + 4 * t * RB);
                to.k[t][NB * W - 2] = a[0];
                to.k[t][NB * W - 1] = a[1];
            }
        }
    }
}
// The loaded registers as operands: block b's in k[t][b * W ..], whose lane group
// g holds elements 8 g .. (fp16), or 16 (g % 2) + 8 (g / 2) .. (int8).
template <bool Q8, int NB> __device__ __forceinline__ void order_k(Tile<Q8, NB> &T) {
    constexpr int RB = 32 * NB * (Q8 ? 1 : 2), UNITS = RB / 128;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) swap_rows(T.k[t][8 * u + i], T.k[t][8 * u + 4 + i]);
        if constexpr (Q8) {
#pragma unroll
            for (int h = 0; h < RB / 64; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) swap_halves(T.k[t][4 * h + i], T.k[t][4 * h + 2 + i]);
        }
    }
}

// lane (m, g): dims 16 n + m, keys 8 g .. 8 g + 7.  int8: one load brings the 16
// tokens of dim 16 n + m for n even in lanes g % 2 == 0 and odd in the others,
// which then change halves.
template <bool Q8, int NB, bool NT>
__device__ __forceinline__ void load_v(Tile<Q8, NB> &to, const uint8_t *mine, int lane) {
    const int m = lane & 15, g = lane >> 4;
    const uint8_t *p = Q8 ? mine + (16 * (g & 1) + m) * 16 : mine + (m * 16 + (g & 1) * 8) * 2;
#pragma unroll
    for (int n = 0; n < (Q8 ? NB : 2 * NB); ++n) {
        const u4 a = load16<NT>(p + n * 512);
#pragma unroll
        for (int i = 0; i < 4; ++i) to.v[4 * n + i] = a[i];
    }
}
template <bool Q8, int NB> __device__ __forceinline__ void order_v(Tile<Q8, NB> &T) {
    if constexpr (Q8) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) swap_odd_rows(T.v[4 * n + i], T.v[4 * n + 2 + i]);
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

// The lane, made anew: for what is seldom done, so that no register keeps anything of it over the tiles.
__device__ __forceinline__ int fresh_lane() {
    int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(lane));
    return lane;
}

// One work-group: a piece of a request's tiles for one kv head and up to
// 16 RT * row_waves of its rows.  Wave w takes the RT row tiles of w % row_waves
// and the tiles w / row_waves + i * (4 / row_waves) of the piece (waves that
// share a key tile read it through the caches); the waves of a row tile join
// through LDS.  With RT = 2 a tile's operands are made once for 32 rows.
template <bool Q8, int NB, bool NT, int RT>
__global__ __launch_bounds__(ATTN_THREADS, ATTN_OCCUPANCY(NB, RT)) void attn_kernel(Cache c, Attn a) {
    constexpr int D = 32 * NB, LD = D + 4;
    // While the tiles go by: q's limbs (operands as lanes read them) and the sums of its blocks, of each wave, or (RT = 2)
    // of each row tile, shared; and each wave's tile's scales.  At the end [wave][16][LD] outputs, then [wave][16] (m, l).
    constexpr int QB = NB * 2 * 1024, QU = QB + (Q8 ? NB * 256 : 0), QPART = QU + (RT > 1 ? 256 : 0), SB = Q8 ? NB * 128 : 0;
    constexpr int JOIN = 16 * (LD + 2) * 4, PART = QPART + SB;
    static_assert(RT == 1 || RT == 2, "four row tiles' limbs in LDS");
    __shared__ __align__(16) uint8_t lds_[ATTN_WAVES * (PART > JOIN ? PART : JOIN)];
    float *lds = (float *)lds_;
    // Priority falls with the tiles done: of a SIMD's waves the oldest issues first, and where loads or vector work queue,
    // the last to come began its tiles only as the first ended (of 32 requests of 8192 tokens, 70 us into 160), and then
    // ran on alone (one request of 65536 Q8_0 tokens and heads of 64 26.9 -> 25.5 us, 8 rows of 4 requests of up to
    // 16384 51 -> 49, one request of 524288 fp16 tokens 334 -> 327).
    __builtin_amdgcn_s_setprio(3);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wg_rows = 16 * RT * a.row_waves, groups = (a.rows_cap + wg_rows - 1) / wg_rows;
    // row groups of a piece (they read the same keys) lie 8 blocks apart: one L2
    const int head = blockIdx.y;
    int item = blockIdx.x, rgroup = 0;
    if (groups > 1) {
        const int per = 8 * groups, oct = item / per, in = item - oct * per;
        item = oct * 8 + (in & 7);
        rgroup = in >> 3;
        if (item >= a.items) return;
    }
    const Req1 r0 = a.items <= a.B ? Req1{0, 0, 0, 0, 0} : attn_req(c, a, lane);
    const int chunk = attn_chunk(c, a, r0, lane);
    const Piece pc = attn_piece(c, a, r0, chunk, item, lane);
    if (pc.b < 0) return;
    if (a.items > a.B && pc.index == 0 && head == 0 && rgroup == 0 && threadIdx.x == 0)
        a.info[pc.b] = int4{pc.whole, pc.last, pc.of, 0};
    const int rows = min(pc.r.n, a.max_q) * a.group;
    const int row0 = rgroup * wg_rows;
    if (row0 >= rows) return;

    const int rw = wave % a.row_waves, kw = wave / a.row_waves, kws = ATTN_WAVES / a.row_waves;
    const int m = lane & 15, g = lane >> 4;
    // a row sees keys [lo, hi); hi_all and lo_all: keys that any row sees, hi_min and lo_max: that every row sees
    const int64_t room = attn_room(c, a);
    const int64_t pos0 = (int64_t)pc.r.ctx - pc.r.n;
    const int hi_all = (int)min((int64_t)pc.r.ctx, room);
    const int hi_min = (int)max(min(pos0 + 1, room), (int64_t)0);
    const int lo_all = a.window ? (int)max(pos0 - a.window + 1, (int64_t)0) : 0;
    const int lo_max = a.window ? (int)max((int64_t)pc.r.ctx - a.window, (int64_t)0) : 0;
    if (((int64_t)pc.r.ctx > room || pc.r.n > a.max_q) && a.err && threadIdx.x == 0) a.err[0] = 1;
    // (of the lane's row of tile i; made where a tile is cut, not kept)
    struct Sight { int lo, hi; };
    auto sight = [&](int i) {
        const int j = div_magic(row0 + 16 * (rw * RT + i) + (fresh_lane() & 15), a.group_magic);
        return Sight{a.window ? (int)max(pos0 + j - a.window + 1, (int64_t)0) : 0, (int)max(min(pos0 + j + 1, room), (int64_t)0)};
    };
    // The q of one row tile (the loads go out first, the limbs are made while the first tile's are on their way): where a
    // wave has two, the waves of the same rows make one each.
    const int qt = RT == 1 ? 0 : kw % RT;
    f4 x[2 * NB];
    bool live;
    {
        const int r = row0 + 16 * (rw * RT + qt) + m, j = div_magic(r, a.group_magic), qh = head * a.group + (r - j * a.group);
        const int64_t trow = (int64_t)pc.r.first + j;
        live = r < rows && trow >= 0 && trow < a.T;
        const float *qp = a.q + (live ? trow * a.ldq + (int64_t)qh * D : 0) + (Q8 ? 16 * (g & 1) + 8 * (g >> 1) : 8 * g);
#pragma unroll
        for (int s = 0; s < NB; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) x[2 * s + e] = *(const f4 *)(qp + 32 * s + 4 * e);
    }

    const int t0 = pc.r.lo + (pc.index ? pc.index * chunk : 0);
    const int t1 = pc.index == pc.of - 1 ? pc.r.lo + pc.r.tiles : t0 + chunk;
    const int first = t0 + kw;
    // (a wave whose rows the request does not have takes no tiles)
    const int N = first < t1 && row0 + 16 * RT * rw < rows ? (t1 - first + kws - 1) / kws : 0;
    const u32 gp = c.page_tokens >> 4, quants = c.page_tokens * D;
    const uint8_t *kb = c.k + (u64)head * c.head_bytes, *vb = c.v + (u64)head * c.head_bytes;
    // Pages of 32 tiles of the wave: lane i holds group i % 2 of tile i / 2, page << 4 | group in page.  The next 32 tiles'
    // table entries are asked for when these are taken up.
    u32 ids = 0, raw = 0;
    uint64_t bad = 0;
    auto group_of = [&](int n, bool *in) {
        const int lane = fresh_lane();
        const int grp = 2 * (first + kws * (n + (lane >> 1))) + (lane & 1);
        *in = n + (lane >> 1) < N && grp * 16 < hi_all && grp * 16 + 16 > lo_all;
        return grp;
    };
    auto ask_ids = [&](int n) {
        bool in;
        const int grp = group_of(n, &in);
        if (in) raw = (u32)a.table[pc.b * a.stride + div_magic(grp, a.gp_magic)];
    };
    auto take_ids = [&](int n) {
        bool in;
        const int grp = group_of(n, &in);
        const bool wrong = in && raw >= c.n_pages;
        ids = in && !wrong ? raw << 4 | ((u32)grp - (u32)div_magic(grp, a.gp_magic) * gp) : 0;
        bad = __ballot(wrong);
        if (wrong && a.err) a.err[0] = 1;
    };
    // Byte offsets of the tile's first 16-token group in K and V alike (quants or halves, and scales), and of the second
    // from there.  (A lane's group is an offset times 0 or 1: chosen between two members of a struct, the compiler put the
    // struct in scratch memory.)
    struct Where { u64 x0, dx, s0, ds; };
    auto where = [&](int n) {
        Where w;
        const u32 i0 = (u32)__builtin_amdgcn_readlane((int)ids, 2 * (n & 31));
        const u32 i1 = (u32)__builtin_amdgcn_readlane((int)ids, 2 * (n & 31) + 1);
        const u64 p0 = (u64)(i0 >> 4) * (u64)c.page_bytes, p1 = (u64)(i1 >> 4) * (u64)c.page_bytes;
        w.x0 = p0 + (i0 & 15) * (16 * D * (Q8 ? 1 : 2));
        w.dx = p1 + (i1 & 15) * (16 * D * (Q8 ? 1 : 2)) - w.x0;
        w.s0 = p0 + quants + (i0 & 15) * (NB * 32);
        w.ds = p1 + quants + (i1 & 15) * (NB * 32) - w.s0;
        return w;
    };
    // V keys of lane (m, g) are in group g / 2; of the scales [K, V][group][block][16] a lane takes the 16 bytes at
    // 16 * (lane % 8 NB)
    const int sl = lane % (8 * NB);
    const uint8_t *sb = (sl / (4 * NB) ? vb : kb) + (sl % (2 * NB)) * 16;
    const bool second = (sl / (2 * NB)) & 1;
    Tile<Q8, NB> T;
    auto get_k = [&](const Where &w) {
        load_k<Q8, NB, NT>(T, kb + w.x0, kb + w.x0 + w.dx, lane);
        if constexpr (Q8) T.s = *(const h8 *)(sb + w.s0 + (second ? w.ds : 0));
    };
    auto get_v = [&](const Where &w) { load_v<Q8, NB, NT>(T, vb + w.x0 + ((g & 2) ? w.dx : 0), lane); };
    auto wrong_of = [&](int n) { return (u32)(bad >> (2 * (n & 31))) & 3; };

    // The first tile's loads, also for a wave without tiles (page 0 then): under a condition, every wait for q behind them
    // would wait for them too.
    ask_ids(0);
    take_ids(0);
    {
        const Where w = where(0);
        get_k(w);
        get_v(w);
        T.wrong = wrong_of(0);
    }
    ask_ids(32);

    // q as two fp16 limbs, in LDS: read again for every tile, they leave their registers to the tile on the way
    auto part = [&](int i) { return lds_ + (RT == 1 ? wave : rw * RT + i) * QPART; };
    float unscale[RT];
    {
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < 2 * NB; ++s) {
            x[s] *= live ? a.scale : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(x[s][k]));
        }
        top = across_groups_max(top);
        int ex = 0;
        if (top > 0.f && top < INFINITY) ex = min(10 - ilogbf(top), 120);
        unscale[0] = ldexpf(1.f, (Q8 ? 24 : 0) - ex);
        if (RT > 1 && kw < RT) *(float *)(part(qt) + QU + lane * 4) = unscale[0];
#pragma unroll
        for (int s = 0; s < NB; ++s) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = ldexpf(x[2 * s + e / 4][e % 4], ex);
            h8 qh, ql;
            limbs(y, &qh, &ql);
            float sum = 0.f;                     // Q8_0: -128 2^-24 times the sum of q's block
            if constexpr (Q8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += (float)qh[e] + (float)ql[e];
                sum = across_groups_sum(sum) * (-128.f / 16777216.f);
            }
            if (RT == 1 || kw < RT) {
                *(h8 *)(part(qt) + (2 * s) * 1024 + lane * 16) = qh;
                *(h8 *)(part(qt) + (2 * s + 1) * 1024 + lane * 16) = ql;
                if constexpr (Q8) *(float *)(part(qt) + QB + s * 256 + lane * 4) = sum;
            }
        }
    }
    if constexpr (RT > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RT; ++i) unscale[i] = *(const float *)(part(i) + QU + lane * 4);
    }

    f4 o[RT][2 * NB];
    float mx[RT], l[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        mx[i] = NONE;
        l[i] = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) o[i][k] = f4{0.f, 0.f, 0.f, 0.f};
    }
    uint8_t *scales = lds_ + ATTN_WAVES * QPART + wave * SB;
    u32 qat = (u32)lane * 16;
    auto is_edge = [&](int tile, u32 wrong) { return wrong || tile * TILE < lo_max || tile * TILE + TILE > hi_min; };
    auto v_half = [&](int k) { return __builtin_bit_cast(h8, u4{T.v[4 * k], T.v[4 * k + 1], T.v[4 * k + 2], T.v[4 * k + 3]}); };
    auto v_scales = [&](int b) { return *(const h8 *)(scales + ((2 + (g >> 1)) * NB + b) * 32 + (g & 1) * 16); };
    // Keys that some rows of the request see and others do not (the newest of several tokens, the oldest of a window): a
    // weight of 0 takes no infinity and no NaN out of the product.  Values that are no numbers (Q8_0: whose product with the
    // scale is none as a half) are taken as 0 in tiles with such keys, and looked up again behind the loop for the rows that
    // see them.  (Looking for them costs 0.1 us a call, 0.2 to 0.4 for Q8_0; the lanes made anew gave back the registers.)
    bool cleared = false;
    auto no_number = [](h8 x, int e) { return (__builtin_bit_cast(us8, x)[e] & 0x7C00) == 0x7C00; };
    // One tile, while the next one's keys and values are asked for.  The last tile is a copy of its own, without these
    // loads: asked for and not used, the barrier behind the loop would wait for them (under a condition, the waits for
    // this tile's values would wait for the next one's keys).
    auto step = [&](int n, auto more) __attribute__((always_inline)) {
        constexpr bool MORE = decltype(more)::value;
        // (q's address is made anew for each tile, so that the reads stay here)
        asm volatile("" : "+v"(qat));
        if constexpr (Q8) *(h8 *)(scales + sl * 16) = T.s;
        // scores of the lane's 8 keys, times 1 / unscale
        order_k<Q8, NB>(T);
        f4 d[RT][2], d2[RT][2];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) d[i][t] = d2[i][t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            h8 k[2], ks;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if constexpr (Q8) k[t] = biased_h8(T.k[t][2 * b], T.k[t][2 * b + 1]);
                else k[t] = __builtin_bit_cast(h8, u4{T.k[t][4 * b], T.k[t][4 * b + 1], T.k[t][4 * b + 2], T.k[t][4 * b + 3]});
            }
            if constexpr (Q8) ks = *(const h8 *)(scales + ((g >> 1) * NB + b) * 32 + (g & 1) * 16);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const h8 qh = *(const h8 *)(part(i) + (2 * b) * 1024 + qat), ql = *(const h8 *)(part(i) + (2 * b + 1) * 1024 + qat);
                if constexpr (Q8) {
                    const float off = *(const float *)(part(i) + QB + b * 256 + (qat >> 2));
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const f4 y = mma(k[t], qh, mma(k[t], ql, f4{off, off, off, off}));
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[i][t][e] = fmaf(y[e], (float)ks[4 * t + e], d[i][t][e]);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        d[i][t] = mma(k[t], qh, d[i][t]);
                        d2[i][t] = mma(k[t], ql, d2[i][t]);
                    }
                }
            }
        }
        const u32 wrong = T.wrong;
        const int tile = first + kws * n;
        Where next;
        if constexpr (MORE) {
            if (((n + 1) & 31) == 0) {
                take_ids(n + 1);
                ask_ids(n + 33);
            }
            next = where(n + 1);
            get_k(next);
            T.wrong = wrong_of(n + 1);
        }
        const bool edge = is_edge(tile, wrong);
        u32 gone = 0;                            // keys of the lane that no row may touch
        if (edge) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int key = tile * TILE + 8 * g + e;
                gone |= (u32)(key >= hi_all || key < lo_all || ((wrong >> (g >> 1)) & 1)) << e;
            }
        }
        h8 ph[RT], pl[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float s[8], p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = Q8 ? d[i][e / 4][e % 4] : d[i][e / 4][e % 4] + d2[i][e / 4][e % 4];
            if (edge) {
                const Sight see = sight(i);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int key = tile * TILE + 8 * g + e;
                    s[e] = ((gone >> e) & 1) || key >= see.hi || key < see.lo ? -INFINITY : s[e];
                }
            }
            float top = s[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
            top *= unscale[i];
            if (__any(top > mx[i] + SLACK)) {
                const float now = fmaxf(mx[i], across_groups_max(top));
                const float keep = __builtin_amdgcn_exp2f(mx[i] - now);
                mx[i] = now;
                l[i] *= keep;
#pragma unroll
                for (int k = 0; k < 2 * NB; ++k) o[i][k] *= keep;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = __builtin_amdgcn_exp2f(fmaf(s[e], unscale[i], LIFT - mx[i]));
                l[i] += p[e];
            }
            limbs(p, &ph[i], &pl[i]);
        }
        order_v<Q8, NB>(T);
        if constexpr (Q8) {
            // (values of their own from here on: as they are changed below, they would else be copied where they are loaded, at
            // the loop's end, with a wait for them)
            if constexpr (RT > 1) {
#pragma unroll
                for (int k = 0; k < 4 * NB; ++k) asm volatile("" : "+v"(T.v[k]));
            }
            bool far = false;                    // a scale is no number, or 512 or more (below, times 128 is a half)
            if (edge && pc.r.n > 1) {
                us8 top = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int b = 0; b < NB; ++b) top = __builtin_elementwise_max(top, __builtin_bit_cast(us8, v_scales(b)));
                const u4 w = __builtin_bit_cast(u4, top);
                u32 any = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32 keep = ((gone >> (2 * i)) & 1 ? 0u : 0x7FFFu) | ((gone >> (2 * i + 1)) & 1 ? 0u : 0x7FFF0000u);
                    any |= (w[i] & keep) + 0x20002000u;
                }
                far = __any((any & 0x80008000u) != 0) != 0;
            }
            if (far) {
                cleared = true;
#pragma unroll
                for (int k = 0; k < 2 * NB; ++k) {
                    h8 vs = v_scales(k / 2);
                    const h8 v = quants_h8(T.v[2 * k], T.v[2 * k + 1]) * vs;
#pragma unroll
                    for (int e = 0; e < 8; ++e) T.v[2 * k + e / 4] &= no_number(v, e) ? ~(0xFFu << (8 * (e & 3))) : ~0u;
                    if (k & 1) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) vs[e] = no_number(vs, e) ? (_Float16)0 : vs[e];
                        *(h8 *)(scales + ((2 + (g >> 1)) * NB + k / 2) * 32 + (g & 1) * 16) = vs;
                    }
                }
            }
            // scale times quant (19 bits, a multiple of 2^-24) is exactly a half and a half's remainder
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                h8 vs = v_scales(b);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) vs[e] = (gone >> e) & 1 ? (_Float16)0 : vs[e];
                }
#pragma unroll
                for (int k = 2 * b; k < 2 * b + 2; ++k) {
                    const h8 v = quants_h8(T.v[2 * k], T.v[2 * k + 1]), vh = v * vs, vl = __builtin_elementwise_fma(v, vs, -vh);
#pragma unroll
                    for (int i = 0; i < RT; ++i) o[i][k] = mma(vh, ph[i], mma(vh, pl[i], mma(vl, ph[i], o[i][k])));
                }
                __builtin_amdgcn_sched_barrier(0);      // (blocks taken further ahead of each other cost registers to scratch)
            }
        } else {
            if (edge) {
                u32 keep[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    keep[i] = ((gone >> (2 * i)) & 1 ? 0u : 0xFFFFu) | ((gone >> (2 * i + 1)) & 1 ? 0u : 0xFFFF0000u);
#pragma unroll
                for (int k = 0; k < 8 * NB; ++k) T.v[k] &= keep[k & 3];
                if (pc.r.n > 1) {
                    const h8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
                    h8 z = zero;                 // stays 0 but for infinities and NaN
#pragma unroll
                    for (int k = 0; k < 2 * NB; ++k) z = __builtin_elementwise_fma(v_half(k), zero, z);
                    const u4 w = __builtin_bit_cast(u4, z);
                    if (__any((w[0] | w[1] | w[2] | w[3]) != 0)) {
                        cleared = true;
#pragma unroll
                        for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
                            for (int e = 0; e < 8; ++e) T.v[4 * k + e / 2] &= no_number(v_half(k), e) ? ~(0xFFFFu << (16 * (e & 1))) : ~0u;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
#pragma unroll
                for (int k = 0; k < 2 * NB; ++k) o[i][k] = mma(v_half(k), ph[i], o[i][k]);
#pragma unroll
                for (int k = 0; k < 2 * NB; ++k) o[i][k] = mma(v_half(k), pl[i], o[i][k]);
            }
        }
        if constexpr (MORE) get_v(next);
    };
    for (int n = 0; n + 1 < N; ++n) {
        if (n == N / 4) __builtin_amdgcn_s_setprio(2);
        if (n == N / 2) __builtin_amdgcn_s_setprio(1);
        if (n == N * 3 / 4) __builtin_amdgcn_s_setprio(0);
        step(n, std::true_type());
    }
    if (N > 0) step(N - 1, std::false_type());
    // outputs of rows that see an infinity or a NaN among the values of such tiles: NaN
    if (cleared) {
        const int g = fresh_lane() >> 4;
        for (int n = 0; n < N; ++n) {
            if ((n & 31) == 0) {
                ask_ids(n);
                take_ids(n);
            }
            const int tile = first + kws * n;
            const u32 wrong = wrong_of(n);
            if (!is_edge(tile, wrong)) continue;
            const Where w = where(n);
            if constexpr (Q8) *(h8 *)(scales + sl * 16) = *(const h8 *)(sb + w.s0 + (second ? w.ds : 0));
            Tile<Q8, NB> P;
            load_v<Q8, NB, NT>(P, vb + w.x0 + ((g & 2) ? w.dx : 0), lane);
            order_v<Q8, NB>(P);
            h8 seen[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const Sight see = sight(i);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int key = tile * TILE + 8 * g + e;
                    seen[i][e] = ((wrong >> (g >> 1)) & 1) || key >= see.hi || key < see.lo ? (_Float16)0 : (_Float16)1;
                }
            }
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k) {
                h8 v, none;
                if constexpr (Q8) v = quants_h8(P.v[2 * k], P.v[2 * k + 1]) * v_scales(k / 2);
                else v = __builtin_bit_cast(h8, u4{P.v[4 * k], P.v[4 * k + 1], P.v[4 * k + 2], P.v[4 * k + 3]});
#pragma unroll
                for (int e = 0; e < 8; ++e) none[e] = no_number(v, e) ? (_Float16)1 : (_Float16)0;
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const f4 count = mma(none, seen[i], f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][k][e] = count[e] > 0.f ? __builtin_nanf("") : o[i][k][e];
                }
            }
        }
    }

    // join the waves of each row tile
    float *stat = lds + ATTN_WAVES * 16 * LD;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        __syncthreads();                         // the place is free (of q's limbs, or the row tiles before)
        l[i] = across_groups_sum(l[i]);
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) *(f4 *)(lds + (wave * 16 + m) * LD + 16 * k + 4 * g) = o[i][k];
        if (g == 0) {
            stat[(wave * 16 + m) * 2] = mx[i];
            stat[(wave * 16 + m) * 2 + 1] = l[i];
        }
        __syncthreads();
        for (int k = threadIdx.x; k < 16 * a.row_waves * (D / 4); k += ATTN_THREADS) {
            const int rr = k / (D / 4), d = (k - rr * (D / 4)) * 4;
            const int row = row0 + 16 * ((rr >> 4) * RT + i) + (rr & 15);
            if (row >= rows) continue;
            float M = NONE, L = 0.f, mw[ATTN_WAVES], lw[ATTN_WAVES];
            f4 x = {0.f, 0.f, 0.f, 0.f}, y[ATTN_WAVES];
#pragma unroll
            for (int w = 0; w < ATTN_WAVES; ++w) {       // (behind the last wave of the keys, the first one's with no weight)
                const int at = ((w < kws ? w * a.row_waves : 0) + (rr >> 4)) * 16 + (rr & 15);
                mw[w] = w < kws ? stat[at * 2] : NONE;
                lw[w] = stat[at * 2 + 1];
                y[w] = *(const f4 *)(lds + at * LD + d);
                M = fmaxf(M, mw[w]);
            }
#pragma unroll
            for (int w = 0; w < ATTN_WAVES; ++w) {
                const float f = w < kws ? __builtin_amdgcn_exp2f(mw[w] - M) : 0.f;
                L = fmaf(f, lw[w], L);
                x += w < kws ? f * y[w] : f4{0.f, 0.f, 0.f, 0.f};
            }
            if (pc.of == 1) {
                const int j = div_magic(row, a.group_magic);
                const int64_t to = (int64_t)pc.r.first + j;
                if (to >= 0 && to < a.T)
                    *(f4 *)(a.out + to * a.ldo + (int64_t)(head * a.group + row - j * a.group) * D + d) =
                        L == 0.f ? f4{0.f, 0.f, 0.f, 0.f} : x * (1.f / L);
            } else {
                const int64_t at = ((int64_t)item * c.kv_heads + head) * a.rows_cap + row;
                *(f4 *)(a.part + at * LD + d) = x;
                if (d == 0) *(f4 *)(a.part + at * LD + D) = f4{M, L, 0.f, 0.f};
            }
        }
    }
}

// Joins the pieces of the requests that were cut: one work-group per row,
// thread (w, d) pieces w, w + WAYS, ... of 4 elements, each with its own running
// m, then the ways through LDS.  A chain of dependent loads is what it takes its
// time for: the request's pieces, then everything else at once.
template <int NB, int THREADS>
__global__ __launch_bounds__(THREADS) void attn_join_kernel(Cache c, Attn a) {
    constexpr int D = 32 * NB, LD = D + 4, LANES = D / 4, WAYS = THREADS / LANES, DEEP = 4;
    __shared__ f4 xs[THREADS];
    __shared__ float ms[WAYS], ls[WAYS];
    const int row = blockIdx.x, head = blockIdx.y, b = blockIdx.z;
    const int first = a.seq_start[b], n = a.seq_start[b + 1] - first;
    const int4 info = a.info[b];                      // (a request without rows has none: left by another call)
    if (n <= 0 || row >= min(n, a.max_q) * a.group || info.z <= 1) return;
    const int pieces = info.z, whole = info.x, last = info.y;
    const int way = threadIdx.x / LANES, d = (threadIdx.x - way * LANES) * 4;
    f4 x = {0.f, 0.f, 0.f, 0.f};
    float M = NONE, L = 0.f;
    if (way < WAYS) {
        for (int i0 = way; i0 < pieces; i0 += DEEP * WAYS) {
            f4 y[DEEP], ml[DEEP];
#pragma unroll
            for (int k = 0; k < DEEP; ++k) {
                const int i = min(i0 + k * WAYS, pieces - 1);
                const int item = i == pieces - 1 ? last : whole + i;
                const float *p = a.part + (((int64_t)item * c.kv_heads + head) * a.rows_cap + row) * LD;
                y[k] = *(const f4 *)(p + d);
                ml[k] = *(const f4 *)(p + D);
            }
#pragma unroll
            for (int k = 0; k < DEEP; ++k) {
                if (i0 + k * WAYS >= pieces) break;
                const float now = fmaxf(M, ml[k][0]);
                const float f = __builtin_amdgcn_exp2f(M - now), h = __builtin_amdgcn_exp2f(ml[k][0] - now);
                M = now;
                L = L * f + ml[k][1] * h;
                x = x * f + y[k] * h;
            }
        }
        if (d == 0) {
            ms[way] = M;
            ls[way] = L;
        }
    }
    xs[threadIdx.x] = x;
    __syncthreads();
    if (way == 0) {
#pragma unroll 4
        for (int w = 1; w < WAYS; ++w) {
            const float now = fmaxf(M, ms[w]);
            const float f = __builtin_amdgcn_exp2f(M - now), h = __builtin_amdgcn_exp2f(ms[w] - now);
            M = now;
            L = L * f + ls[w] * h;
            x = x * f + xs[w * LANES + threadIdx.x] * h;
        }
        const int j = div_magic(row, a.group_magic);
        const int64_t to = (int64_t)first + j;
        if (to >= 0 && to < a.T)
            *(f4 *)(a.out + to * a.ldo + (int64_t)(head * a.group + row - j * a.group) * D + d) =
                L == 0.f ? f4{0.f, 0.f, 0.f, 0.f} : x * (1.f / L);
    }
}

template <int NB> int launch_attn(bool q8, bool nt, int rt, const Cache &c, const Attn &a, hipStream_t st);

} // namespace kv
} // namespace kq
