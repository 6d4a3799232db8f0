"""The paged key-value cache operators in plain numpy and 64 bits, written from
include/kqkv.h alone: the page layout, the quantisation of a block, the plan of
a step, rotary positions and the attention."""
import numpy as np

F16, Q8_0 = 1, 8


def quantise(x):
    """fp32 [..., 32] blocks -> int8 quants, fp16 scales."""
    x = np.asarray(x, dtype=np.float32)
    m = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    with np.errstate(all="ignore"):
        s = np.minimum(m * (np.float32(1) / np.float32(127)), np.float32(65504)).astype(np.float16)
        f = s.astype(np.float32)[..., None]
        n = np.where(f > 0, np.rint(x / f), 0)
    n = np.where(bad[..., None], 0, np.clip(n, -127, 127)).astype(np.int8)
    return n, np.where(bad, np.float16(np.nan), s)


class Cache:
    """K and V as the bytes of n_pages pages; fresh memory is NaN."""

    def __init__(self, type, heads, dim, page, n_pages):
        self.type, self.heads, self.dim, self.page, self.n_pages = type, heads, dim, page, n_pages
        n = page * dim
        self.head_bytes = 2 * n if type == F16 else n + n // 16
        self.k = np.full((n_pages, heads, self.head_bytes), 0x7E, dtype=np.uint8)   # 0x7E7E: an fp16 NaN
        self.v = self.k.copy()

    def _views(self, b):
        n = self.page * self.dim
        if self.type == F16:
            return b.view(np.float16), None
        return b[:, :, :n].view(np.int8), b[:, :, n:].view(np.float16)

    def _at(self, t, v):
        d = np.arange(self.dim)
        return (t // 16) * 16 * self.dim + d * 16 + t % 16 if v else t * self.dim + d

    def _scale_at(self, t):
        b = np.arange(self.dim // 32)
        return (t // 16) * (self.dim // 32) * 16 + b * 16 + t % 16

    def put(self, slot, k, v):
        """k, v: fp32 [heads][dim]."""
        p, t = divmod(int(slot), self.page)
        for b, x, is_v in ((self.k, k, False), (self.v, v, True)):
            e, s = self._views(b)
            if self.type == F16:
                with np.errstate(over="ignore"):
                    e[p][:, self._at(t, is_v)] = np.asarray(x, dtype=np.float32).astype(np.float16)
            else:
                q, sc = quantise(np.asarray(x).reshape(self.heads, -1, 32))
                e[p][:, self._at(t, is_v)] = q.reshape(self.heads, self.dim)
                s[p][:, self._scale_at(t)] = sc

    def get(self, slot):
        """The exact values of a slot, fp64 [heads][dim] of K and of V."""
        p, t = divmod(int(slot), self.page)
        out = []
        for b, is_v in ((self.k, False), (self.v, True)):
            e, s = self._views(b)
            x = e[p][:, self._at(t, is_v)].astype(np.float64)
            if self.type != F16:
                x = x * np.repeat(s[p][:, self._scale_at(t)].astype(np.float64), 32, axis=1)
            out.append(x)
        return out

    def fill(self, rng, table, lens):
        """Random values for the tokens of each request."""
        for row, n in zip(table, lens):
            for i in range(n):
                slot = int(row[i // self.page]) * self.page + i % self.page
                self.put(slot, rng.standard_normal((self.heads, self.dim)), rng.standard_normal((self.heads, self.dim)))


def plan(ctx, new, page, table, held, free, n_pages, n_free, T):
    """The step of kqkv_plan: a dict of its outputs (copies)."""
    B, stride = table.shape
    r = dict(table=table.copy(), held=held.copy(), free=free.copy(), n_free=n_free, slots=np.full(T, -1, np.int32),
             pos=np.zeros(T, np.int32), start=np.zeros(B + 1, np.int32), ctx=ctx.copy(), err=0)
    fail = dict(r, err=1)
    if n_free < 0 or (ctx < 0).any() or (held < 0).any() or (held > stride).any():
        return fail
    top = n_free
    ends = [b for b in range(B) if new[b] < 0]
    gone = sum(int(held[b]) for b in ends)
    need = {b: max(0, -(-(int(ctx[b]) + int(new[b])) // page) - int(held[b])) for b in range(B) if new[b] >= 0}
    if top + gone > n_pages or sum(need.values()) > top + gone or sum(max(0, int(n)) for n in new) > T:
        return fail
    if any(int(held[b]) + n > stride for b, n in need.items()):
        return fail
    if any(-(-(int(ctx[b]) + int(new[b])) // page) > stride for b in need):
        return fail
    free, table = r["free"].copy(), r["table"]
    for b in ends:
        for j in range(held[b]):
            free[top] = table[b, j]
            top += 1
        r["held"][b] = r["ctx"][b] = 0
    r["free"] = free.copy()
    t = 0
    for b in range(B):
        r["start"][b] = t
        if new[b] < 0:
            continue
        for j in range(need[b]):
            top -= 1
            table[b, held[b] + j] = free[top]
        r["held"][b] = held[b] + need[b]
        r["ctx"][b] = ctx[b] + new[b]
        for i in range(new[b]):
            p = int(ctx[b]) + i
            id = int(table[b, p // page])
            r["pos"][t], r["slots"][t] = p, id * page + p % page if 0 <= id < n_pages else -1
            t += 1
    r["start"][B] = t
    r["n_free"] = top
    return r


def rope(x, pos, style, rot, base, sections, factors=None):
    """x [T][heads][dim] at pos [axes][T]: fp64, unrounded."""
    y = np.asarray(x, dtype=np.float64).copy()
    axis = np.repeat(np.arange(len(sections)), sections)
    i = np.arange(rot // 2)
    f = np.float64(np.float32(base)) ** (-2.0 * i / rot)
    if factors is not None:
        f = f / np.asarray(factors, dtype=np.float64)
    t = (np.asarray(pos, dtype=np.float64)[axis].T * f)[:, None, :]
    a, b = (i, i + rot // 2) if style == 0 else (2 * i, 2 * i + 1)
    va, vb = y[:, :, a].copy(), y[:, :, b].copy()
    y[:, :, a] = va * np.cos(t) - vb * np.sin(t)
    y[:, :, b] = va * np.sin(t) + vb * np.cos(t)
    return y


def attn(cache, table, ctx, start, q, q_heads, scale, window, max_q=8, out=None):
    """Rows of `out` (or zeros) with the requests' rows filled in, and the size
    of each output's error bound, fp64.

    The bound, for u = 2^-24: q enters in two fp16 limbs, 22 bits, so within
    2^-21 of its row's largest magnitude's products; the products' sum over dim
    elements in fp32 adds at most dim * u of sum |q k|.  A score is then off by at
    most e = A (2^-21 + dim u), A = scale * max|q| sum |k| (largest over
    the keys), a weight by e + 2^-21 (exp2 and its limbs) of itself, numerator and
    denominator alike; their sums run over at most n / 32 + 64 additions.  So
    |error| <= 2 (e + 2^-21 + (n / 32 + 64) u) * sum w |v| / sum w.
    (A weight below 2^-9 of the largest is off by up to 2^-31 of the largest, n
    2^-31 max|v| over a row: within the n 2^-28 of the additions' term as long as
    max|v| is at most 8 times the weighted mean of |v|.)"""
    T = q.shape[0]
    kv, d, page = cache.heads, cache.dim, cache.page
    g = q_heads // kv
    o = np.zeros((T, q_heads, d)) if out is None else np.array(out, dtype=np.float64).reshape(T, q_heads, d)
    tol = np.zeros_like(o)
    q = np.asarray(q, dtype=np.float64).reshape(T, q_heads, d)
    u = 2.0 ** -24
    for b in range(len(ctx)):
        n = int(start[b + 1]) - int(start[b])
        c = max(0, int(ctx[b]))
        rows = [(j, int(start[b]) + j) for j in range(min(n, max_q)) if 0 <= int(start[b]) + j < T]
        if not rows:
            continue
        there, ks, vs = [], [], []
        for i in range(min(c, table.shape[1] * page)):
            id = int(table[b, i // page])
            if 0 <= id < cache.n_pages:
                k, v = cache.get(id * page + i % page)
                there.append(i)
                ks.append(k)
                vs.append(v)
        there = np.array(there, dtype=np.int64)
        for j, r in rows:
            p = c - n + j
            seen = (there <= p) & ((there > p - window) if window else True)
            o[r] = 0
            if not seen.any():
                continue
            k = np.stack(ks)[seen]
            v = np.stack(vs)[seen]
            for h in range(q_heads):
                s = scale * (k[:, h // g] @ q[r, h])
                w = np.exp(s - s.max())
                o[r, h] = w @ v[:, h // g] / w.sum()
                A = abs(scale) * np.abs(q[r, h]).max() * np.abs(k[:, h // g]).sum(1).max()
                e = A * (2.0 ** -21 + d * u) + 2.0 ** -21 + (len(s) / 32 + 64) * u
                tol[r, h] = 2 * e * (w @ np.abs(v[:, h // g])) / w.sum()
    return o.reshape(T, -1), tol.reshape(T, -1)
