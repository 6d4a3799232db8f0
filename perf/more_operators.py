"""The operators of one decode or verify step that stand beside the products and the cache:

  norm    the residual's addition and the root-mean-square norm of rows or heads, as fp32 rows and as Q8_0 blocks (a fp16 scale
          for 32 int8 quants)
  moe     a whole mixture-of-experts layer for 1 to 8 tokens: router, choice of experts, gate and up products, activation, down
          product and weighted sum, the experts' weights packed in GGUF blocks
  sample  one token for each row of logits, with temperature, top-k, top-p and min-p, from given random numbers

`run` computes them with elementary torch operations, or, where `own` is true, with the library's calls.
"""
import math
import random

import torch

own = False

Q4_0, Q8_0, Q2_K, Q3_K, Q4_K, Q5_K, Q6_K = 2, 8, 10, 11, 12, 13, 14
# weights of a block, its bytes, where its fp16 scale and minimum are, and the spread of (scale * quant) with the other bits random
BLOCKS = {Q4_0: (32, 18, 0, None, 4.6), Q8_0: (32, 34, 0, None, 74.0), Q2_K: (256, 84, 80, 82, 13.0), Q3_K: (256, 110, 108, None, 42.0),
          Q4_K: (256, 144, 0, 2, 190.0), Q5_K: (256, 176, 0, 2, 380.0), Q6_K: (256, 210, 208, None, 1370.0)}
MEAN_QUANT = {Q2_K: 1.5, Q4_K: 7.5, Q5_K: 15.5}  # a block's minimum is about this many of its scales


# ---- cases --------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # the next token of one request: latency alone (hidden size of the 30B mixture-of-experts shapes)
        dict(name="norm: 1 token of 2048", op="norm", tokens=1, heads=1, n=2048, add=True, pad=0, f32=True, q8=False),
        # the heads of a verify batch's queries, between the projection and the rotary positions, inside the fused q, k, v rows
        dict(name="norm: 250 tokens, 32 heads of 128", op="norm", tokens=250, heads=32, n=128, add=False, pad=1024, f32=True, q8=False),
        # a prompt chunk at the 8B shapes, the normed rows also in 8 bits
        dict(name="norm: 4099 tokens of 4096, q8_0", op="norm", tokens=4099, heads=1, n=4096, add=True, pad=0, f32=True, q8=True),
        # a long prompt chunk at the 70B shapes
        dict(name="norm: 8192 tokens of 8192", op="norm", tokens=8192, heads=1, n=8192, add=True, pad=0, f32=True, q8=False),
        # a layer of the 30B mixture-of-experts shapes, one token of one request
        dict(name="moe: 1 token, 8 of 128", op="moe", tokens=1, E=128, k=8, hidden=2048, inner=768, gate=Q4_K, down=Q6_K,
             score="softmax", renorm=True, bias=False, scale=1.0, act="silu", add=True),
        # the same for a verify pass of eight positions
        dict(name="moe: 8 tokens, 8 of 128", op="moe", tokens=8, E=128, k=8, hidden=2048, inner=768, gate=Q4_K, down=Q6_K,
             score="softmax", renorm=True, bias=False, scale=1.0, act="silu", add=True),
        # a small layer of odd sizes in the simple 32-weight blocks
        dict(name="moe: 5 tokens, 2 of 11, q8_0", op="moe", tokens=5, E=11, k=2, hidden=608, inner=1184, gate=Q8_0, down=Q4_0,
             score="softmax", renorm=False, bias=False, scale=1.0, act="gelu", add=False),
        # a wide layer whose router scores each expert by itself and chooses with a bias
        dict(name="moe: 3 tokens, 6 of 160, sigmoid", op="moe", tokens=3, E=160, k=6, hidden=5120, inner=1536, gate=Q5_K, down=Q4_K,
             score="sigmoid", renorm=True, bias=True, scale=2.5, act="silu", add=True),
        # the next token of one chat, with the usual settings
        dict(name="sample: 1 row of 32000", op="sample", rows=1, V=32000, pad=0, mix="usual"),
        # a verify pass of eight positions over a large vocabulary, each with settings of its own
        dict(name="sample: 8 rows of 128256", op="sample", rows=8, V=128256, pad=0, mix="each"),
        # a large serving batch; odd vocabulary, some rows with most tokens masked
        dict(name="sample: 256 rows of 151937", op="sample", rows=256, V=151937, pad=0, mix="each"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "moe", "moe", "moe", "sample", "sample"])
    if op == "norm":
        if rng.random() < 0.4:
            heads, n = rng.choice([(32, 128), (64, 128), (8, 64), (5, 256), (9, 96), (1, 32), (16, 80), (71, 64)])
        else:
            heads, n = 1, 4 * _log(rng, 16, 4096)
        q8 = n % 32 == 0 and rng.random() < 0.4
        return dict(op=op, tokens=min(_log(rng, 1, 8192), (1 << 25) // (heads * n) + 1), heads=heads, n=n, add=rng.random() < 0.6,
                    pad=rng.choice([0, 0, 4, 1024]), f32=not q8 or rng.random() < 0.7, q8=q8)
    if op == "moe":
        simple = rng.random() < 0.25
        step = 32 if simple else 256
        kinds = [Q4_0, Q8_0] if simple else [Q2_K, Q3_K, Q4_K, Q4_K, Q5_K, Q6_K, Q8_0, Q4_0]
        k = rng.choice([1, 2, 2, 4, 6, 8, 8, 10, 16])
        hidden, inner = step * (_log(rng, 256, 5120) // step), step * (_log(rng, 256, 2048) // step)
        return dict(op=op, tokens=rng.randint(1, 8), E=max(k, _log(rng, 4, 256)), k=k, hidden=hidden, inner=inner, gate=rng.choice(kinds),
                    down=rng.choice(kinds), score=rng.choice(["softmax", "softmax", "sigmoid"]), renorm=rng.random() < 0.7,
                    bias=rng.random() < 0.3, scale=rng.choice([1.0, 1.0, 2.5]), act=rng.choice(["silu", "silu", "gelu"]),
                    add=rng.random() < 0.6)
    V = _log(rng, 500, 200000)
    return dict(op=op, rows=min(_log(rng, 1, 256), 30000000 // V), V=V, pad=rng.choice([0, 0, 0, 1, 64]), mix=rng.choice(["usual", "each", "each", "plain", "greedy"]))


def _row_bytes(kind, n):
    return n // BLOCKS[kind][0] * BLOCKS[kind][1]


def work(case):
    if case["op"] == "norm":
        n = case["tokens"] * case["heads"] * case["n"]
        q8 = n // 32 * 34 if case["q8"] else 0
        return {"bytes": n * 4 * (1 + 2 * case["add"] + case["f32"]) + q8 * 2 + (n * 4 if q8 else 0) + 4 * case["n"],
                "flops": n * (4 + case["add"])}
    if case["op"] == "moe":
        t, E, k, h, f = (case[x] for x in ("tokens", "E", "k", "hidden", "inner"))
        distinct = E * (1 - (1 - k / E) ** t)  # experts that t tokens choose between them
        each = 2 * f * _row_bytes(case["gate"], h) + h * _row_bytes(case["down"], f)
        return {"bytes": int(distinct * each) + E * h * 4 + t * h * 4 * (2 + case["add"]) + t * k * 8, "flops": 2 * t * (k * 3 * h * f + E * h)}
    return {"bytes": case["rows"] * (case["V"] * 4 + 28), "flops": case["rows"] * case["V"] * 4}


# ---- inputs -------------------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    s = {"norm": _prepare_norm, "moe": _prepare_moe, "sample": _prepare_sample}[case["op"]](case, _gen(seed))
    s["case"] = case
    return s


def _prepare_norm(case, g):
    t, w, pad = case["tokens"], case["heads"] * case["n"], case["pad"]
    x = torch.randn(t, w + pad, device="cuda", generator=g)
    x *= torch.exp(torch.randn(t, 1, device="cuda", generator=g))  # tokens of different size, a few channels far larger
    x[:, torch.randint(0, w, (3,), device="cuda", generator=g)] *= 30
    s = dict(x=x[:, :w], gain=1 + 0.3 * torch.randn(case["n"], device="cuda", generator=g), eps=1e-6)
    if case["add"]:
        s["add"] = 0.5 * torch.randn(t, w, device="cuda", generator=g)
    s["sum"], s["y"] = torch.empty(t, w, device="cuda") if case["add"] else None, torch.empty(t, w, device="cuda") if case["f32"] else None
    if case["q8"]:
        s["y8"] = torch.empty(t * w // 32 * 34, dtype=torch.uint8, device="cuda")
        s["back"] = torch.empty(t, w, device="cuda")
    return s


def _packed(kind, rows, n, g):
    """rows x n weights of spread n^-1/2 in packed blocks: every field random, scales within a factor of three."""
    qk, size, at, at_min, spread = BLOCKS[kind]
    blocks = rows * (n // qk)
    out = torch.randint(0, 256, (blocks, size), dtype=torch.uint8, device="cuda", generator=g)
    d = (0.5 + torch.rand(blocks, device="cuda", generator=g)) * (n ** -0.5 / spread)
    out[:, at:at + 2] = d.half().view(torch.uint8).view(blocks, 2)
    if at_min is not None:
        low = d * MEAN_QUANT[kind] * (0.8 + 0.4 * torch.rand(blocks, device="cuda", generator=g))
        out[:, at_min:at_min + 2] = low.half().view(torch.uint8).view(blocks, 2)
    return out.view(-1)


def _prepare_moe(case, g):
    t, E, k, h, f = (case[x] for x in ("tokens", "E", "k", "hidden", "inner"))
    x = torch.randn(t, h, device="cuda", generator=g)
    s = dict(x=x, router=torch.randn(E, h, device="cuda", generator=g) * (1.5 * h ** -0.5), y=torch.empty(t, h, device="cuda"),
             ids=torch.empty(t, k, dtype=torch.int32, device="cuda"), route=torch.empty(t, k, device="cuda"),
             bias=0.1 * torch.randn(E, device="cuda", generator=g) if case["bias"] else None,
             add=torch.randn(t, h, device="cuda", generator=g) if case["add"] else None,
             gate=_packed(case["gate"], E * f, h, g), up=_packed(case["gate"], E * f, h, g), down=_packed(case["down"], E * h, f, g))
    if own:
        import dequant_gemv_gguf_amd as kq
        s["layer"] = kq.MoELayer(E, k, h, f, case["gate"], s["gate"], s["up"], case["down"], s["down"], s["router"], s["bias"],
                                 kq.KQSTEP_SOFTMAX if case["score"] == "softmax" else kq.KQSTEP_SIGMOID, case["renorm"], case["scale"],
                                 kq.KQSTEP_SILU if case["act"] == "silu" else kq.KQSTEP_GELU)
        s["ws"] = torch.empty(kq.kqstep_moe_workspace_bytes(s["layer"], t), dtype=torch.uint8, device="cuda")
    return s


def _prepare_sample(case, g):
    m, V = case["rows"], case["V"]
    wide = torch.randn(m, V + case["pad"], device="cuda", generator=g) * 2.5  # what follows a row in its buffer is not a logit
    logits = wide[:, :V]
    hot = torch.randint(0, V, (m, 24), device="cuda", generator=g)
    logits.scatter_add_(1, hot, 9 * torch.rand(m, 24, device="cuda", generator=g))
    if case["mix"] == "each":
        for i in range(m):
            if i % 5 == 3:  # a grammar leaves few tokens
                logits[i].masked_fill_(torch.rand(V, device="cuda", generator=g) < 0.95, -math.inf if i % 2 else torch.finfo(torch.float32).min)
            if i % 64 == 61:
                logits[i] = -math.inf  # ... or none
    pick = lambda v, dtype: torch.tensor(v, dtype=dtype, device="cuda")[torch.randint(0, len(v), (m,), device="cuda", generator=g)].contiguous()  # noqa: E731
    f, i = torch.float32, torch.int32
    if case["mix"] == "usual":
        r = dict(temperature=pick([0.8], f), top_k=pick([40], i), top_p=pick([0.95], f), min_p=pick([0.05], f))
    elif case["mix"] == "each":
        r = dict(temperature=pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.5], f), top_k=pick([0, 0, 1, 20, 50, 1000], i), top_p=pick([1.0, 0.5, 0.9, 0.95, 0.99], f),
                 min_p=pick([0.0, 0.0, 0.02, 0.1], f))
    elif case["mix"] == "plain":
        r = dict(temperature=pick([0.7, 1.0, 1.3], f), top_k=None, top_p=None, min_p=None)
    else:
        r = dict(temperature=pick([0.0], f), top_k=None, top_p=None, min_p=None)
    s = dict(logits=logits, u=torch.rand(m, device="cuda", generator=g), tokens=torch.empty(m, dtype=i, device="cuda"), probs=torch.empty(m, device="cuda"), **r)
    if own:
        import dequant_gemv_gguf_amd as kq
        s["ws"] = torch.empty(kq.kqstep_sample_workspace_bytes(m, V), dtype=torch.uint8, device="cuda")
    return s


# ---- the operators ------------------------------------------------------------------------------------------------------

def run(s):
    return {"norm": _norm, "moe": _moe, "sample": _sample}[s["case"]["op"]](s)


def _norm(s):
    c = s["case"]
    t, heads, n = c["tokens"], c["heads"], c["n"]
    w = heads * n
    if own:
        import dequant_gemv_gguf_amd as kq
        kq.kqstep_norm(t, heads, n, s["x"], s["x"].stride(0), s.get("add"), w, s["sum"], w, s["gain"], s["eps"], s["y"], w, s.get("y8"))
        if c["q8"]:
            kq.kq_dequant(Q8_0, s["y8"], t * w, s["back"])
        return [v for v in (s["sum"], s["y"], s.get("back")) if v is not None]
    h = s["x"] + s["add"] if c["add"] else s["x"]
    h64 = h.reshape(t, heads, n).double()
    y = (h64 * s["gain"].double() * torch.rsqrt((h64 * h64).mean(-1, keepdim=True) + s["eps"])).float().reshape(t, w)
    out = [h] if c["add"] else []
    if c["f32"]:
        out.append(y)
    if c["q8"]:
        b = y.view(t, -1, 32)
        d = (b.abs().amax(-1) / 127).half().float()[..., None]
        out.append((torch.where(d > 0, torch.round(b / d), 0).clamp(-127, 127) * d).view(t, w))
    return out


def _nibbles(q, n):
    """Bytes [..., 32 * n] -> 4-bit quants [..., 64 * n]: 32 low nibbles, then their 32 high ones."""
    q = q.unflatten(-1, (n, 1, 32))
    return torch.cat([q & 15, q >> 4], -2).flatten(-3)


def _six_bit(b):
    """The 12 packed bytes of Q4_K and Q5_K -> 8 scales and 8 minima."""
    low, mid, high = b[..., 0:4], b[..., 4:8], b[..., 8:12]
    return torch.cat([low & 63, (high & 15) | ((low >> 6) << 4)], -1), torch.cat([mid & 63, (high >> 4) | ((mid >> 6) << 4)], -1)


def _dequant(kind, rows, n):
    """Packed rows (uint8 [..., bytes]) -> fp32 weights [..., n]."""
    qk, size, at, at_min, _ = BLOCKS[kind]
    b = rows.reshape(-1, size)
    d = b[:, at:at + 2].contiguous().view(torch.float16).float()
    low = b[:, at_min:at_min + 2].contiguous().view(torch.float16).float() if at_min is not None else None
    if kind == Q8_0:
        w = d * b[:, 2:].contiguous().view(torch.int8).float()
    elif kind == Q4_0:
        w = d * (torch.cat([b[:, 2:] & 15, b[:, 2:] >> 4], -1).float() - 8)
    elif kind in (Q4_K, Q5_K):
        sc, mn = _six_bit(b[:, 4:16])
        q = _nibbles(b[:, -128:], 4)
        if kind == Q5_K:
            bit = torch.arange(8, device=b.device, dtype=torch.uint8)[:, None]
            q = q + (((b[:, None, 16:48] >> bit) & 1) << 4).flatten(1)
        w = ((d * sc.float())[..., None] * q.view(-1, 8, 32).float() - (low * mn.float())[..., None]).flatten(1)
    elif kind == Q6_K:
        sc = b[:, 192:208].contiguous().view(torch.int8).float()
        ql, qh = b[:, :128].reshape(-1, 2, 64), b[:, 128:192].reshape(-1, 2, 32)
        low4 = torch.cat([ql & 15, ql >> 4], -1)
        high2 = torch.cat([(qh >> s) & 3 for s in (0, 2, 4, 6)], -1)
        w = ((d * sc)[..., None] * ((low4 | (high2 << 4)).view(-1, 16, 16).float() - 32)).flatten(1)
    else:  # 2 low bits: 32 bytes hold 128 quants
        part = b[:, 16:80] if kind == Q2_K else b[:, 32:96]
        part = part.reshape(-1, 2, 32)
        q = torch.stack([(part >> s) & 3 for s in (0, 2, 4, 6)], 2).view(-1, 16, 16).float()
        if kind == Q2_K:
            w = ((d * (b[:, :16] & 15).float())[..., None] * q - (low * (b[:, :16] >> 4).float())[..., None]).flatten(1)
        else:
            s8 = b[:, 96:104]
            four = torch.cat([s8 & 15, s8 >> 4], -1)
            two = torch.cat([(b[:, 104:108] >> s) & 3 for s in (0, 2, 4, 6)], -1)
            sc = (four | (two << 4)).float() - 32
            bit = torch.stack([(b[:, :32] >> j) & 1 for j in range(8)], 1).view(-1, 16, 16).float()
            w = ((d * sc)[..., None] * (q - 4 * (1 - bit))).flatten(1)
    return w.view(*rows.shape[:-1], n)


def _moe(s):
    c = s["case"]
    t, E, k, h, f = (c[x] for x in ("tokens", "E", "k", "hidden", "inner"))
    if own:
        import dequant_gemv_gguf_amd as kq
        kq.kqstep_moe(s["layer"], t, s["x"], h, s["add"], h, s["y"], h, s["ids"], s["route"], s["ws"], s["ws"].numel())
        return s["y"], s["ids"], s["route"]
    logits = torch.matmul(s["x"].double(), s["router"].double().t())  # the choice must not turn on a rounding
    score = torch.softmax(logits, -1) if c["score"] == "softmax" else torch.sigmoid(logits)
    ids = torch.sort(score + s["bias"].double() if c["bias"] else logits, descending=True, stable=True)[1][:, :k]
    p = score.gather(1, ids)
    if c["renorm"]:
        p = p / p.sum(-1, keepdim=True)
    p = (p * c["scale"]).float()
    at = ids.reshape(-1)
    x = s["x"].repeat_interleave(k, 0)[..., None]
    part = lambda w, kind, rows, n: _dequant(kind, w.view(E, rows, -1)[at], n)  # noqa: E731
    gate = torch.matmul(part(s["gate"], c["gate"], f, h), x)
    up = torch.matmul(part(s["up"], c["gate"], f, h), x)
    if c["act"] == "silu":
        inner = gate / (1 + torch.exp(-gate)) * up
    else:
        inner = 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))) * up
    out = torch.matmul(part(s["down"], c["down"], h, f), inner).view(t, k, h)
    y = (out * p[..., None]).sum(1)
    return y + s["add"] if c["add"] else y, ids.to(torch.int32), p


def _sample(s):
    c = s["case"]
    m, V = c["rows"], c["V"]
    if own:
        import dequant_gemv_gguf_amd as kq
        kq.kqstep_sample(m, V, s["logits"], s["logits"].stride(0), s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], s["tokens"], s["probs"],
                         s["ws"], s["ws"].numel())
        return s["tokens"], s["probs"]
    l = torch.where(torch.isnan(s["logits"]), -math.inf, s["logits"])
    l, order = torch.sort(l, descending=True, stable=True)
    top = l[:, :1]
    t = s["temperature"].double()[:, None]
    w = torch.where(l == top, 1.0, torch.exp((l.double() - top.double()) / torch.where(t > 0, t, 1)))
    w = torch.where((l == -math.inf) | ((t <= 0) & (torch.arange(V, device="cuda") > 0)), 0, w)
    keep = w > 0
    if s["top_k"] is not None:
        top_k = s["top_k"][:, None]
        keep &= (torch.arange(V, device="cuda") < top_k) | (top_k <= 0)
        w = torch.where(keep, w, 0)
    if s["top_p"] is not None:
        top_p, cum = s["top_p"].double()[:, None], w.cumsum(-1)
        keep &= (cum - w < top_p * cum[:, -1:]) | (top_p >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    keep[:, 0] = top[:, 0] > -math.inf
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0))  # in the order of the vocabulary
    cum = kept.cumsum(-1)
    total = cum[:, -1:]
    at = (cum > s["u"].double()[:, None] * total).to(torch.int8).argmax(-1, keepdim=True)
    p = (kept.gather(1, at) / torch.where(total > 0, total, 1)).float()[:, 0]
    return torch.where(total > 0, at, -1).to(torch.int32)[:, 0], p


# ---- the same in 64 bits ------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "moe": _exact_moe, "sample": _exact_sample}[case["op"]](s)


def _exact_norm(s):
    c = s["case"]
    t, heads, n = c["tokens"], c["heads"], c["n"]
    out = []
    rows, sums = torch.empty(t, heads * n, dtype=torch.float64, device="cuda"), None
    x = s["x"].double()
    if c["add"]:
        sums = x + s["add"].double()
        x = sums.float().double()  # the norm is that of the row as it goes on
    for i in range(heads):
        part = x[:, i * n:(i + 1) * n]
        size = torch.linalg.vector_norm(part, dim=1)
        rows[:, i * n:(i + 1) * n] = part / torch.sqrt(size ** 2 / n + s["eps"])[:, None] * s["gain"].double()
    out = [sums] if c["add"] else []
    if c["f32"]:
        out.append(rows)
    if c["q8"]:  # blocks are made of the 32-bit values
        b = rows.float().double().view(-1, 32)
        step = (b.abs().max(1).values.float() / 127).half().double()
        q = torch.zeros_like(b)
        some = step > 0
        q[some] = (b[some] / step[some, None]).round().clamp(-127, 127) * step[some, None]
        out.append(q.view(t, -1))
    return out


def _element_maps(kind):
    """For each weight of a block: where its bits lie (byte, shift, width, place), which are added up."""
    bits = []
    for e in range(BLOCKS[kind][0]):
        j, half, l = e // 32, e // 128, e % 32
        if kind == Q8_0:
            m = [(2 + e, 0, 8, 0)]
        elif kind == Q4_0:
            m = [(2 + e % 16, 4 * (e // 16), 4, 0)]
        elif kind in (Q4_K, Q5_K):
            m = [((16 if kind == Q4_K else 48) + 32 * (e // 64) + l, 4 * (j % 2), 4, 0)]
            if kind == Q5_K:
                m.append((16 + l, j, 1, 4))
        elif kind == Q6_K:
            m = [(64 * half + 32 * (j % 2) + l, 4 * (j % 4 // 2), 4, 0), (128 + 32 * half + l, 2 * (j % 4), 2, 4)]
        elif kind == Q2_K:
            m = [(16 + 32 * half + l, 2 * (j % 4), 2, 0)]
        else:
            m = [(32 + 32 * half + l, 2 * (j % 4), 2, 0), (l, j, 1, 2)]
        bits.append(m)
    return bits


def _exact_weights(kind, packed, n):
    """Packed rows -> 64-bit weights, weight by weight from where its bits lie."""
    qk, size, at, at_min, _ = BLOCKS[kind]
    b = packed.reshape(-1, size).to(torch.int32)
    half = lambda o: packed.reshape(-1, size)[:, o:o + 2].contiguous().view(torch.float16).double()  # noqa: E731
    maps = _element_maps(kind)
    q = 0
    for part in range(len(maps[0])):
        byte, shift, width, place = (torch.tensor([m[part][i] for m in maps], device="cuda") for i in range(4))
        q = q + (((b[:, byte] >> shift) & ((1 << width) - 1)) << place)
    q = q.double()
    if kind == Q8_0:
        w = half(0) * torch.where(q > 127, q - 256, q)
    elif kind == Q4_0:
        w = half(0) * (q - 8)
    elif kind in (Q4_K, Q5_K):
        cols = []
        for j in range(8):
            if j < 4:
                cols.append((b[:, 4 + j] & 63, b[:, 8 + j] & 63))
            else:
                cols.append(((b[:, 8 + j] & 15) + 16 * (b[:, j] >> 6), (b[:, 8 + j] >> 4) + 16 * (b[:, 4 + j] >> 6)))
        sc, mn = (torch.stack([c[i] for c in cols], 1).repeat_interleave(32, 1).double() for i in (0, 1))
        w = half(0) * sc * q - half(2) * mn
    elif kind == Q6_K:
        sc = b[:, 192:208].repeat_interleave(16, 1)
        w = half(208) * torch.where(sc > 127, sc - 256, sc).double() * (q - 32)
    elif kind == Q2_K:
        sm = b[:, :16].repeat_interleave(16, 1)
        w = half(80) * (sm & 15).double() * q - half(82) * (sm >> 4).double()
    else:
        cols = []
        for i in range(16):
            four = b[:, 96 + i % 8] >> (4 * (i // 8)) & 15
            cols.append(four + 16 * ((b[:, 104 + i % 4] >> (2 * (i // 4))) & 3) - 32)
        w = half(108) * torch.stack(cols, 1).repeat_interleave(16, 1).double() * (q - 4)
    return w.reshape(-1, n)


def _exact_moe(s):
    c = s["case"]
    E, k, h, f = (c[x] for x in ("E", "k", "hidden", "inner"))
    y, route = torch.zeros_like(s["x"], dtype=torch.float64), torch.zeros(c["tokens"], k, dtype=torch.float64, device="cuda")
    for t in range(c["tokens"]):
        x = s["x"][t].double()
        logits = [float(v) for v in (s["router"].double() * x).sum(1)]
        if c["score"] == "softmax":
            most = max(logits)
            total = math.fsum(math.exp(v - most) for v in logits)
            score = [math.exp(v - most) / total for v in logits]
        else:
            score = [1 / (1 + math.exp(-v)) for v in logits]
        by = [a + b for a, b in zip(score, s["bias"].tolist())] if c["bias"] else logits
        chosen = sorted(range(E), key=lambda e: (-by[e], e))[:k]
        share = math.fsum(score[e] for e in chosen) if c["renorm"] else 1.0
        for j, e in enumerate(chosen):
            gate, up = (_exact_weights(c["gate"], s[n].view(E, -1)[e], h) @ x for n in ("gate", "up"))
            if c["act"] == "silu":
                inner = gate * torch.sigmoid(gate) * up
            else:  # (1 + tanh z) / 2 is the logistic function of 2 z
                inner = gate * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate * gate * gate)) * up
            route[t, j] = score[e] / share * c["scale"]
            y[t] += route[t, j] * (_exact_weights(c["down"], s["down"].view(E, -1)[e], f) @ inner)
        if c["add"]:
            y[t] += s["add"][t].double()
    return y, None, route


def _exact_sample(s):
    """The probability of each row's token (the tokens are whole numbers)."""
    c = s["case"]
    out = torch.zeros(c["rows"], dtype=torch.float64)
    setting = lambda name, i, none: none if s[name] is None else float(s[name][i])  # noqa: E731
    for i in range(c["rows"]):
        l = s["logits"][i].double()
        there = ((l == l) & (l != -math.inf)).nonzero()[:, 0]
        if not len(there):
            continue
        t, k, p, low = (setting(*a) for a in (("temperature", i, 1.0), ("top_k", i, 0), ("top_p", i, 1.0), ("min_p", i, 0.0)))
        if t <= 0:
            out[i] = 1
            continue
        l = l[there]
        if 0 < k < len(l):  # every token above the k-th largest logit, and as many of those that equal it as are left
            edge = l.kthvalue(len(l) - int(k) + 1).values
            equal = (l == edge).nonzero()[:, 0][:int(k) - int((l > edge).sum())]
            stay = l > edge
            stay[equal] = True
            l = l[stay]
        w = torch.exp((l - l.max()) / t)
        down, at = torch.sort(-w, stable=True)
        down = -down
        n = len(w)
        if p < 1:
            n = min(n, int((down.cumsum(0) < p * float(w.sum())).sum()) + 1)
        n = max(1, min(n, int((down >= low).sum())))
        kept = torch.zeros_like(w)
        kept[at[:n]] = down[:n]
        cum = kept.cumsum(0)
        at = int(torch.searchsorted(cum, float(s["u"][i]) * cum[-1], right=True))
        out[i] = kept[at] / cum[-1]
    return None, out.cuda()
