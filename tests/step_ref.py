"""The operators of include/kqstep.h in plain numpy and 64 bits, written from the
header alone; products of packed weights come from the oracle."""
import numpy as np

import kqsynth
import oracle

F32 = np.float32


def norm(x, add, heads, weight, eps):
    """x, add [T][heads * n] -> h (fp32, exactly what has to come) and y (64 bits)."""
    with np.errstate(all="ignore"):
        h = x if add is None else (x + add).astype(F32)
        p = h.astype(np.float64).reshape(len(h), heads, -1)
        w = 1.0 if weight is None else weight.astype(np.float64)
        y = p * w / np.sqrt((p * p).mean(-1, keepdims=True) + float(F32(eps)))
    return h, y.reshape(h.shape)


def check_norm(y, want):
    """y is the fp32 nearest to want, but for 64-bit roundings (a sum of up to 2^20 squares, a root, two products: below 2^-40) that
    decide between two of them: half a step, and half the smallest one."""
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(y - want) <= np.abs(want) * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -149)
        both = (np.isnan(y) & np.isnan(want)) | (y == want)
        big = (np.abs(want) > 3.4028235e38) & np.isinf(y)
    assert not (bad & ~both & ~big).any(), np.abs(y - want)[bad & ~both & ~big].max()


def route(x, router, bias, k, score, renorm, scale):
    """One token: ids, weights (64 bits)."""
    with np.errstate(all="ignore"):
        l = (router.astype(np.float64) * x.astype(np.float64)).sum(1)
        if score == 0:
            s = np.exp(l - np.nanmax(l))
            s = s / s.sum()
        else:
            s = 1 / (1 + np.exp(-l))
        by = l if bias is None else s + bias.astype(np.float64)
        order = sorted(range(len(l)), key=lambda e: (by[e] != by[e], -by[e] if by[e] == by[e] else 0, e))[:k]
        p = s[order]
        if renorm:
            p = p / p.sum()
    return order, p * float(F32(scale))


def act(kind, g):
    if kind == 0:
        return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def moe(c, x, add):
    """c: dict of a layer (numpy).  Returns y, ids, weights, and how far y may be off when every product is within the documented
    1e-4 sum |w x| + 1e-6 of the exact one: an error d of g moves act(g) by at most 1.13 d (the slopes of both activations stay below
    that), errors of inner go through |down|; sums and products of fp32 roundings are far below these."""
    E, k, H, F = c["E"], c["k"], c["hidden"], c["inner"]
    T = len(x)
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    ids, weights = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        ids[t], weights[t] = route(x[t], c["router"], c["bias"], k, c["score"], c["renorm"], c["scale"])
        for e, p in zip(ids[t], weights[t]):
            (g, sg), (u, su) = (oracle.gemv(c["gate_type"], c[n][e], F, H, x[t:t + 1]) for n in ("gate", "up"))
            dg, du = 1e-4 * sg[0] + 1e-6, 1e-4 * su[0] + 1e-6
            a = act(c["act"], g[0])
            inner = a * u[0]
            d_inner = 1.13 * dg * (np.abs(u[0]) + du) + np.abs(a) * du + 2.0 ** -21 * np.abs(inner)
            w = oracle.dequant(c["down_type"], c["down"][e], H * F).reshape(H, F).astype(np.float64)
            y[t] += p * (w @ inner)
            tol[t] += abs(p) * (np.abs(w) @ (d_inner + 1e-4 * np.abs(inner)) + 1e-6)
    if add is not None:
        y += add
        tol += 2.0 ** -20 * np.abs(add)
    return y, ids, weights, tol


def layer(rng, E, k, hidden, inner, gate_type, down_type, score=0, renorm=True, bias=False, scale=1.0, act=0):
    """Random weights; scales such that gate and up products of unit activations are of the order of one."""
    def packed(kind, rows, n):
        qk, size, at, at_min = kqsynth.BLOCK[kind]
        b = kqsynth.blocks(kind, E * rows * (n // qk), rng)
        spread = {2: 4.6, 8: 74, 10: 13, 11: 42, 12: 190, 13: 380, 14: 1370}[kind]
        d = (n ** -0.5 / spread * rng.uniform(0.5, 1.5, len(b))).astype(np.float16)
        b[:, at:at + 2] = d.view(np.uint8).reshape(-1, 2)
        if at_min is not None:
            m = (d * F32({10: 1.5, 12: 7.5, 13: 15.5}[kind])).astype(np.float16)
            b[:, at_min:at_min + 2] = m.view(np.uint8).reshape(-1, 2)
        return b.reshape(E, rows, -1)
    return dict(E=E, k=k, hidden=hidden, inner=inner, gate_type=gate_type, down_type=down_type, score=score, renorm=renorm,
                scale=scale, act=act, gate=packed(gate_type, inner, hidden), up=packed(gate_type, inner, hidden),
                down=packed(down_type, hidden, inner), router=(rng.standard_normal((E, hidden)) * 1.5 * hidden ** -0.5).astype(F32),
                bias=(0.1 * rng.standard_normal(E)).astype(F32) if bias else None)


def sample(l, t, top_k, top_p, min_p, u):
    """One row: token, its probability (64 bits), and the number of tokens kept."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    there = np.nonzero(l > -np.inf)[0]
    if not len(there):
        return -1, 0.0, 0
    order = there[np.lexsort((there, -l[there]))]
    top = l[order[0]]
    if not t > 0:
        return int(order[0]), 1.0, 1
    with np.errstate(all="ignore"):
        w = np.where(l[order] == top, 1.0, np.exp((l[order] - top) / float(F32(t))))
        w[np.isnan(w)] = 0
    n = len(order)
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        cum = np.cumsum(w[:n])
        n = min(n, int((cum < float(F32(top_p)) * cum[-1]).sum()) + 1)
    if min_p > 0:
        n = min(n, max(1, int((w >= float(F32(min_p))).sum())))
    kept = np.zeros(len(l))
    kept[order[:n]] = w[:n]
    cum = np.cumsum(kept)
    at = int(np.searchsorted(cum, min(max(float(F32(u)), 0.0), 1 - 2.0 ** -24) * cum[-1], side="right"))
    return at, kept[at] / cum[-1], n
