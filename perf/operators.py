"""The operators around a paged key-value cache, as one decode or verify step calls them between the projections:

  plan    pages taken and given back, slots, positions and row offsets of the step's new tokens, from the requests' lengths
  store   rotary positions (one or several axes) on q and k, and k and v put into the cache's pages (fp16, or 8-bit blocks of 32 with an fp16 scale)
  attn    attention of each request's 1 to 8 new tokens over its pages

`run` computes them with elementary torch operations, or, where `own` is true, with the library's calls.

A cache page holds `page` tokens of every key-value head, head after head.  Of one head it holds, for K, the tokens' rows
[page][dim], and for V, groups of 16 tokens [page / 16][dim][16]; an 8-bit page has int8 quants there and after them their
fp16 scales, [page / 16][dim / 32][16] for both.
"""
import math
import random

import torch

own = False

F16, Q8_0 = "f16", "q8_0"


# ---- cases --------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # every request of a small serving batch gets its next token
        dict(name="plan: 16 requests, one token", op="plan", seqs=16, min_ctx=1, max_ctx=4096, new=1, page=16, lens=1),
        # a large batch takes in prompts beside its decoding requests: tens of thousands of new tokens
        dict(name="plan: 256 requests, prompts", op="plan", seqs=256, min_ctx=0, max_ctx=16384, new=4096, page=64, lens=2),
        # a single request's next token (32 q heads, hidden 4096)
        dict(name="store: one token, f16", op="store", tokens=1, heads=32, kv_heads=8, dim=128, page=16, type=F16,
             style="halves", rot=128, axes=1, base=500000.0, factors=True, far=8192, fused=False),
        # a verify pass of a batch at the 70B shapes (64 q heads, hidden 8192), far positions
        dict(name="store: 250 tokens, q8_0", op="store", tokens=250, heads=64, kv_heads=8, dim=128, page=32, type=Q8_0,
             style="pairs", rot=128, axes=1, base=10000.0, factors=False, far=1000000, fused=False),
        # a chunk of a prompt with images: positions in time, height and width
        dict(name="store: 4099 tokens, f16, 3 axes", op="store", tokens=4099, heads=32, kv_heads=4, dim=128, page=16, type=F16,
             style="halves", rot=128, axes=3, base=1000000.0, factors=False, far=32768, fused=True),
        # a long prompt chunk into an 8-bit cache, rotation over a part of each head
        dict(name="store: 8192 tokens, q8_0", op="store", tokens=8192, heads=64, kv_heads=8, dim=128, page=64, type=Q8_0,
             style="halves", rot=64, axes=1, base=10000.0, factors=False, far=131072, fused=False),
        # the first tokens of a chat: latency alone
        dict(name="attn: 1 request, 37 tokens, f16", op="attn", seqs=1, min_ctx=37, max_ctx=37, new=1, heads=32, kv_heads=8, dim=128,
             page=16, type=F16, window=0, lens=3),
        # one long document, one token at a time: all of the card on one request
        dict(name="attn: 1 request, 131072, f16", op="attn", seqs=1, min_ctx=131072, max_ctx=131072, new=1, heads=64, kv_heads=8, dim=128,
             page=16, type=F16, window=0, lens=4),
        # a ragged serving batch
        dict(name="attn: 32 requests, 8192, f16", op="attn", seqs=32, min_ctx=100, max_ctx=8192, new=1, heads=64, kv_heads=8, dim=128,
             page=64, type=F16, window=0, lens=5),
        # every query head with its own key-value head, sliding window, odd lengths
        dict(name="attn: 24 requests, window, f16", op="attn", seqs=24, min_ctx=1, max_ctx=9001, new=1, heads=16, kv_heads=16, dim=64,
             page=16, type=F16, window=1000, lens=6),
        # a verify pass of eight positions over an 8-bit cache
        dict(name="attn: 4 requests, verify 8, q8_0", op="attn", seqs=4, min_ctx=5000, max_ctx=16384, new=8, heads=64, kv_heads=8, dim=128,
             page=32, type=Q8_0, window=0, lens=7),
        # the largest: a full batch of long ragged requests over an 8-bit cache
        dict(name="attn: 64 requests, 32768, q8_0", op="attn", seqs=64, min_ctx=2000, max_ctx=32768, new=1, heads=64, kv_heads=8, dim=128,
             page=64, type=Q8_0, window=0, lens=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "store", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 48, 64, 128])
    lens = rng.randrange(1 << 30)
    if op == "plan":
        seqs = _log(rng, 1, 256)
        c = dict(op=op, seqs=seqs, min_ctx=rng.choice([0, 1, 100]), max_ctx=_log(rng, 100, 16384), new=rng.choice([1, 1, 8, _log(rng, 8, 4096)]), page=page, lens=lens)
        return c
    heads, kv_heads, dim = rng.choice([(64, 8, 128), (32, 8, 128), (32, 4, 128), (16, 16, 64), (28, 4, 128), (8, 1, 256), (12, 2, 96), (9, 3, 64), (71, 1, 64), (10, 5, 32)])
    kind = rng.choice([F16, Q8_0])
    if op == "store":
        rot = rng.choice([dim, dim, dim // 2])
        axes = rng.choice([1, 1, 3, 4])
        return dict(op=op, tokens=_log(rng, 1, 4099 if heads > 32 else 8192), heads=heads, kv_heads=kv_heads, dim=dim, page=page, type=kind,
                    style=rng.choice(["halves", "pairs"]), rot=rot, axes=axes, base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    factors=rng.random() < 0.3, far=_log(rng, 1000, 1000000), fused=rng.random() < 0.5)
    most = 1 << 19 if kind == Q8_0 else 1 << 18  # tokens in all
    max_ctx = _log(rng, 1, 131072)
    seqs = min(_log(rng, 1, 64), max(1, most * 128 * 8 // (dim * kv_heads * max_ctx)))
    return dict(op=op, seqs=seqs, min_ctx=max(1, min(max_ctx, rng.choice([1, 50, max_ctx // 2, max_ctx]))), max_ctx=max_ctx,
                new=rng.choice([1, 1, 1, 2, 5, 8]), heads=heads, kv_heads=kv_heads, dim=dim, page=page, type=kind,
                window=rng.choice([0, 0, 0, _log(rng, 16, 8192)]), lens=lens)


def _lens(case):
    """The requests' lengths before the step (attn: with its new tokens): spread over their logarithm, the first the longest."""
    r = random.Random(case["lens"])
    lo, hi = case["min_ctx"], case["max_ctx"]
    return [hi if i == 0 else int(round(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1))) - 1)) for i in range(case["seqs"])]


def _new(case):
    """New tokens of each request.  plan: some requests end (-1), some wait (0)."""
    r = random.Random(case["lens"] + 1)
    if case["op"] == "attn":
        return [min(n, case["new"] if i == 0 else r.randint(1, case["new"])) for i, n in enumerate(_lens(case))]
    return [case["new"] if i == 0 else -1 if r.random() < 1 / 16 else 0 if r.random() < 1 / 16 else
            1 if r.random() < 0.5 else r.randint(1, case["new"]) for i in range(case["seqs"])]


def _page_bytes(case):
    n = case["kv_heads"] * case["page"] * case["dim"]
    return 2 * n if case["type"] == F16 else n + n // 16


def work(case):
    if case["op"] == "plan":
        lens, new, p = _lens(case), _new(case), case["page"]
        total = sum(max(n, 0) for n in new)
        pages = sum(-(-(a + n) // p) - -(-a // p) if n >= 0 else -(-a // p) for a, n in zip(lens, new))
        return {"bytes": 4 * (3 * len(lens) + 3 * len(lens) + 2 * pages + 2 * total), "flops": 0}
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    per = 2 * kv * d * (2 if case["type"] == F16 else 1 + 1 / 16)  # a token's cache bytes
    if case["op"] == "store":
        t = case["tokens"]
        out = t * 2 * kv * d * 4 if case["type"] == Q8_0 else 0  # what is held in 8 bits is read back
        return {"bytes": t * (h * d * 8 + 2 * kv * d * 4 + per + 4 * case["axes"] + 4) + (out + t * per if out else 0), "flops": t * (h + kv) * case["rot"] * 3}
    keys = flops = rows = 0
    for n, q in zip(_lens(case), _new(case)):
        w = min(n, case["window"] + q - 1) if case["window"] else n
        keys += w
        rows += q
        flops += 4 * q * h * d * w
    return {"bytes": int(keys * per + rows * h * d * 8 + 4 * keys / case["page"]), "flops": flops}


# ---- inputs -------------------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    s = {"plan": _prepare_plan, "store": _prepare_store, "attn": _prepare_attn}[case["op"]](case, seed)
    s["case"] = case
    return s


def _tables(lens, page, spare, width, g):
    """A table of shuffled pages, and the list of the pages that nobody holds."""
    held = [-(-n // page) for n in lens]
    order = torch.randperm(sum(held) + spare, device="cuda", generator=g).to(torch.int32)
    h = _ints(held)
    col = torch.arange(width, device="cuda")
    mine = col < h[:, None]
    at = (h.cumsum(0) - h)[:, None] + col
    table = torch.where(mine, order[at.clamp(max=order.numel() - 1)], -1).to(torch.int32).contiguous()
    return h, table, order[sum(held):].contiguous(), order.numel()


def _prepare_plan(case, seed):
    g = _gen(seed)
    lens, new, page = _lens(case), _new(case), case["page"]
    width = -(-(case["max_ctx"] + case["new"]) // page) + 1
    spare = sum(-(-(a + max(n, 0)) // page) for a, n in zip(lens, new)) + 7
    held, table, left, pages = _tables(lens, page, spare, width, g)
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:left.numel()] = left
    total = sum(max(n, 0) for n in new)
    rows = -(-total // 16) * 16
    e = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(ctx=_ints(lens), new=_ints(new), table=table, held=held, held_out=e(len(lens)), free=free, n_free=_ints([left.numel()]),
                n_free_out=e(1), slots=e(rows), pos=e(rows), start=e(len(lens) + 1), ctx_out=e(len(lens)), err=e(1), rows=rows)


def _prepare_store(case, seed):
    g = _gen(seed)
    t, h, kv, d, page = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    gain = torch.exp(0.5 * torch.randn(kv * d, device="cuda", generator=g))  # keys have channels of their own size
    if case["fused"]:  # one buffer of q, k and v side by side
        all_ = torch.randn(t, (h + 2 * kv) * d, device="cuda", generator=g)
        q, k, v = all_[:, :h * d], all_[:, h * d:(h + kv) * d], all_[:, (h + kv) * d:]
        k *= gain
    else:
        q = torch.randn(t, h * d, device="cuda", generator=g)
        k = torch.randn(t, kv * d, device="cuda", generator=g) * gain
        v = torch.randn(t, kv * d, device="cuda", generator=g)
    first = int(torch.randint(0, page, (1,), device="cuda", generator=g))  # the tokens begin inside a page
    pages = -(-t // page) + 2
    i = first + torch.arange(t, device="cuda")
    slots = (torch.randperm(pages, device="cuda", generator=g)[i // page] * page + i % page).to(torch.int32)
    if t > 20:
        slots[-3:] = -1  # rows that pad the batch
    far = int(torch.randint(0, case["far"], (1,), device="cuda", generator=g))
    pos = [far + torch.arange(t, device="cuda"), far + torch.arange(t, device="cuda") // 32, far + torch.arange(t, device="cuda") % 32, torch.arange(t, device="cuda") // 7]
    pos = torch.stack(pos[:case["axes"]]).to(torch.int32).contiguous()
    pairs = case["rot"] // 2
    sections = [pairs] if case["axes"] == 1 else [pairs - (case["axes"] - 1) * (pairs // 4)] + [pairs // 4] * (case["axes"] - 1)
    factors = 1 + 7 * torch.rand(pairs, device="cuda", generator=g) if case["factors"] else None
    kb, vb = (torch.zeros(pages + 1, _page_bytes(case), dtype=torch.uint8, device="cuda") for _ in range(2))  # the last page takes nothing of use
    s = dict(q=q, k=k, v=v, slots=slots, pos=pos, sections=sections, factors=factors, kb=kb, vb=vb, pages=pages, q_out=torch.empty(t, h * d, device="cuda"),
             k_rows=torch.zeros(t, kv * d, device="cuda"), v_rows=torch.zeros(t, kv * d, device="cuda"))
    if own:
        import dequant_gemv_gguf_amd as kq
        s["cache"] = kq.KVCache(kq.KQKV_F16 if case["type"] == F16 else kq.KQKV_Q8_0, kv, d, page, pages, kb, vb)
        s["rope"] = kq.KVRope(kq.KQKV_ROPE_HALVES if case["style"] == "halves" else kq.KQKV_ROPE_PAIRS, case["rot"], case["base"], sections, factors)
    return s


def _prepare_attn(case, seed):
    g = _gen(seed)
    lens, new, page, kv, d = _lens(case), _new(case), case["page"], case["kv_heads"], case["dim"]
    width = -(-max(lens) // page)
    held, table, _, pages = _tables(lens, page, 3, width, g)
    # what a page holds beside its request's tokens is left from before: here, NaN
    used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    ctx = _ints(lens)
    at = torch.arange(width * page, device="cuda").view(width, page)
    mine = table >= 0
    used[table[mine].long()] = (at < ctx[:, None, None])[mine]
    kb, vb = (torch.empty(pages, _page_bytes(case), dtype=torch.uint8, device="cuda") for _ in range(2))
    if case["type"] == F16:
        k = torch.randn(pages, kv, page, d, device="cuda", dtype=torch.float16, generator=g)
        k.masked_fill_(~used[:, None, :, None], math.nan)
        kb.copy_(k.view(pages, -1).view(torch.uint8))
        del k
        v = torch.randn(pages, kv, page // 16, d, 16, device="cuda", dtype=torch.float16, generator=g)
        v.masked_fill_(~used.view(pages, 1, page // 16, 1, 16), math.nan)
        vb.copy_(v.view(pages, -1).view(torch.uint8))
        del v
    else:
        for b in (kb, vb):
            x = b.view(pages, kv, -1)
            x.copy_(torch.randint(0, 256, x.shape, device="cuda", dtype=torch.uint8, generator=g))
            scale = ((0.5 + torch.rand(pages, kv, page // 16, d // 32, 16, device="cuda", generator=g)) / 73).half()
            scale.masked_fill_(~used.view(pages, 1, page // 16, 1, 16), math.nan)
            x[:, :, page * d:] = scale.view(pages, kv, -1).view(torch.uint8)
            x[:, :, :page * d].masked_fill_(x[:, :, :page * d] == 128, 127)
    rows = sum(new)
    q = torch.randn(rows, case["heads"] * d, device="cuda", generator=g)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = dict(kb=kb, vb=vb, table=table, ctx=ctx, start=_ints(start), q=q, out=torch.zeros_like(q), rows=rows, width=width, err=_ints([0]))
    if own:
        import dequant_gemv_gguf_amd as kq
        s["cache"] = kq.KVCache(kq.KQKV_F16 if case["type"] == F16 else kq.KQKV_Q8_0, kv, d, page, pages, kb, vb)
        n = kq.kqkv_attn_workspace_bytes(s["cache"], len(lens), case["new"], case["max_ctx"], case["heads"])
        s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return s


# ---- the operators ------------------------------------------------------------------------------------------------------

def run(s):
    return {"plan": _plan, "store": _store, "attn": _attn}[s["case"]["op"]](s)


def _plan(s):
    c = s["case"]
    if own:
        import dequant_gemv_gguf_amd as kq
        kq.kqkv_plan(c["seqs"], s["ctx"], s["new"], c["page"], s["table"], s["table"].shape[1], s["held"], s["held_out"], s["free"], s["free"].numel(),
                     s["n_free"], s["n_free_out"], s["rows"], s["slots"], s["pos"], s["start"], s["ctx_out"], s["err"])
        return {k: s[k] for k in ("table", "held_out", "free", "n_free_out", "slots", "pos", "start", "ctx_out", "err")}
    p, table, free, rows = c["page"], s["table"], s["free"], s["rows"]
    ctx, new, held, width = s["ctx"].long(), s["new"].long(), s["held"].long(), s["table"].shape[1]
    ends = new < 0
    more = new.clamp(min=0)
    after = torch.where(ends, 0, ctx + more)
    pages = (after + p - 1) // p
    need = torch.where(ends, 0, (pages - held).clamp(min=0))
    gone = torch.where(ends, held, 0)
    top = s["n_free"].long() + gone.sum()
    ok = (need.sum() <= top) & (more.sum() <= rows) & (pages <= width).all() & (top <= free.numel())
    col = torch.arange(width, device="cuda")
    # the pages of requests that end go on top of the list, in order
    back = ends[:, None] & (col < held[:, None]) & ok
    to = torch.where(back, s["n_free"].long() + (gone.cumsum(0) - gone)[:, None] + col, free.numel()).clamp(max=free.numel())
    wide = torch.cat([free, free.new_zeros(1)])
    wide[to.reshape(-1)] = table.reshape(-1)
    free = wide[:-1]
    # the others take theirs from the top
    take = (col >= held[:, None]) & (col < (held + need)[:, None]) & ok
    at = top - 1 - ((need.cumsum(0) - need)[:, None] + col - held[:, None])
    table = torch.where(take, free[at.clamp(0, free.numel() - 1)], table)
    start = torch.cat([more.new_zeros(1), more.cumsum(0)]) * ok
    i = torch.arange(rows, device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), i, right=True).clamp(max=c["seqs"] - 1)
    live = i < start[-1]
    pos = torch.where(live, ctx[b] + i - start[b], 0)
    slot = torch.where(live, table[b, (pos // p).clamp(max=width - 1)].long() * p + pos % p, -1)
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(table=table, held_out=i32(torch.where(ok, torch.where(ends, 0, held + need), held)), free=free,
                n_free_out=i32(torch.where(ok, top - need.sum(), s["n_free"])), slots=i32(slot), pos=i32(pos), start=i32(start),
                ctx_out=i32(torch.where(ok, after, ctx)), err=i32(torch.where(ok, s["err"], 1)))


def _rotate(x, cos, sin, heads, dim, rot, style):
    """Rotary positions on rows of `heads` heads, in 64 bits, rounded once."""
    x = x.reshape(-1, heads, dim).double()
    y = x.clone()
    if style == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    return y.float()


def _store(s):
    c = s["case"]
    t, h, kv, d, page = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    if own:
        import dequant_gemv_gguf_amd as kq
        kq.kqkv_rope_store(s["cache"], s["rope"], t, s["pos"], t, s["slots"], h, s["q"], s["q"].stride(0), s["q_out"], h * d,
                           s["k"], s["k"].stride(0), s["v"], s["v"].stride(0))
        if c["type"] == Q8_0:
            kq.kqkv_load(s["cache"], t, s["slots"], s["k_rows"], s["v_rows"])
            return s["q_out"], s["k_rows"], s["v_rows"]
        return s["q_out"], s["kb"][:-1].view(torch.float16), s["vb"][:-1].view(torch.float16)
    pairs = torch.arange(c["rot"] // 2, device="cuda")
    freq = torch.pow(c["base"], -2.0 * pairs.double() / c["rot"])
    if s["factors"] is not None:
        freq = freq / s["factors"].double()
    axis = sum((pairs >= sum(s["sections"][:n])).long() for n in range(1, c["axes"])) if c["axes"] > 1 else torch.zeros_like(pairs)
    angle = (s["pos"].double().t()[:, axis] * freq)[:, None]
    cos, sin = angle.cos(), angle.sin()
    q = _rotate(s["q"], cos, sin, h, d, c["rot"], c["style"])
    k = _rotate(s["k"], cos, sin, kv, d, c["rot"], c["style"])
    v = s["v"].reshape(t, kv, d)
    slot = torch.where(s["slots"] >= 0, s["slots"].long(), s["pages"] * page)
    p, at = slot // page, slot % page
    if c["type"] == F16:
        s["kb"].view(torch.float16).view(-1, kv, page, d)[p, :, at] = k.half()
        s["vb"].view(torch.float16).view(-1, kv, page // 16, d, 16)[p, :, at // 16, :, at % 16] = v.half()
        return q.reshape(t, -1), s["kb"][:-1].view(torch.float16), s["vb"][:-1].view(torch.float16)
    kq8, kd = _blocks(k)
    vq8, vd = _blocks(v)
    both = []
    for b, x, dd in ((s["kb"], kq8, kd), (s["vb"], vq8, vd)):
        b = b.view(-1, kv, page * d + page * d // 16)
        quants, scales = b[:, :, :page * d].view(torch.int8), b[:, :, page * d:].view(torch.float16).view(-1, kv, page // 16, d // 32, 16)
        if b.data_ptr() == s["kb"].data_ptr():
            quants = quants.view(-1, kv, page, d)
            quants[p, :, at] = x
        else:
            quants = quants.view(-1, kv, page // 16, d, 16)
            quants[p, :, at // 16, :, at % 16] = x
        scales[p, :, at // 16, :, at % 16] = dd
        both.append(torch.where((s["slots"] >= 0)[:, None, None], (x.float().view(t, kv, -1, 32) * dd.float()[..., None]).view(t, kv, d), 0).reshape(t, -1))
    return q.reshape(t, -1), both[0], both[1]


def _blocks(x):
    """Blocks of 32: an fp16 scale of a 127th of the largest magnitude, and the nearest multiples of that scale."""
    b = x.reshape(x.shape[0], x.shape[1], -1, 32)
    d = (b.abs().amax(-1) / 127).half()
    f = d.float()[..., None]
    n = torch.where(f > 0, torch.round(b / f), 0).clamp(-127, 127)
    return n.to(torch.int8).reshape(x.shape), d


def _pages(s, table):
    """Keys and values of the pages in `table` [requests][n] as 32-bit [requests][kv][n * page][dim]."""
    c = s["case"]
    kv, d, page = c["kv_heads"], c["dim"], c["page"]
    b, n = table.shape
    at = table.clamp(min=0).long()
    if c["type"] == F16:
        k = s["kb"].view(torch.float16).view(-1, kv, page, d)[at].float()
        v = s["vb"].view(torch.float16).view(-1, kv, page // 16, d, 16)[at].float()
    else:
        def parts(x):
            x = x.view(-1, kv, page * d + page * d // 16)[at]
            return x[..., :page * d].view(torch.int8).float(), x[..., page * d:].contiguous().view(torch.float16).float().view(b, n, kv, page // 16, d // 32, 16)
        k, ks = parts(s["kb"])
        k = (k.view(b, n, kv, page, d // 32, 32) * ks.transpose(-1, -2).reshape(b, n, kv, page, d // 32, 1)).view(b, n, kv, page, d)
        v, vs = parts(s["vb"])
        v = (v.view(b, n, kv, page // 16, d // 32, 32, 16) * vs[..., None, :]).view(b, n, kv, page // 16, d, 16)
    k = k.permute(0, 2, 1, 3, 4).reshape(b, kv, n * page, d)
    v = v.permute(0, 2, 1, 3, 5, 4).reshape(b, kv, n * page, d)
    return k, v


def _attn(s):
    c = s["case"]
    h, kv, d, most = c["heads"], c["kv_heads"], c["dim"], c["new"]
    if own:
        import dequant_gemv_gguf_amd as kq
        kq.kqkv_attn(s["cache"], c["seqs"], most, c["max_ctx"], s["ctx"], s["start"], s["table"], s["width"], h, s["rows"], s["q"], h * d,
                     1 / math.sqrt(d), c["window"], s["out"], h * d, s["ws"], s["ws"].numel(), s["err"])
        return s["out"]
    g, ctx, start = h // kv, s["ctx"].long(), s["start"].long()
    k, v = _pages(s, s["table"])
    key = torch.arange(k.shape[2], device="cuda")
    there = (key < ctx[:, None])[:, None, :, None]
    k, v = torch.where(there, k, 0), torch.where(there, v, 0)
    j = torch.arange(most, device="cuda")
    row = (start[:-1, None] + j).clamp(max=s["rows"] - 1)
    q = s["q"].view(-1, kv, g, d)[row].permute(0, 2, 1, 3, 4).reshape(c["seqs"], kv, most * g, d)
    score = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    at = ctx[:, None] - (start[1:] - start[:-1])[:, None] + j
    seen = key <= at[..., None]
    if c["window"]:
        seen &= key > at[..., None] - c["window"]
    seen = seen[:, None, :, None].expand(-1, kv, -1, g, -1).reshape(score.shape)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(torch.isfinite(top), top, 0))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, 1)
    o = o.view(c["seqs"], kv, most, g, d).permute(0, 2, 1, 3, 4)
    t = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return o[b, t - start[b]].reshape(s["rows"], h * d)


# ---- the same in 64 bits ------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_store(s) if case["op"] == "store" else _exact_attn(s)


def _exact_store(s):
    c = s["case"]
    t, h, kv, d, page, rot = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"], c["rot"]
    axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    turn = torch.empty(t, rot // 2, dtype=torch.complex128, device="cuda")
    for i in range(rot // 2):
        f = c["base"] ** (-2 * i / rot) / (float(s["factors"][i]) if s["factors"] is not None else 1.0)
        turn[:, i] = torch.exp(1j * (s["pos"][axis[i]].double() * f))

    def rotated(x, heads):
        x = x.reshape(t, heads, d).double()
        first = [i if c["style"] == "halves" else 2 * i for i in range(rot // 2)]
        second = [i + rot // 2 if c["style"] == "halves" else 2 * i + 1 for i in range(rot // 2)]
        z = torch.complex(x[:, :, first], x[:, :, second]) * turn[:, None]
        x[:, :, first], x[:, :, second] = z.real, z.imag
        return x

    q, k, v = rotated(s["q"], h), rotated(s["k"], kv), s["v"].reshape(t, kv, d).double()
    slots = s["slots"].tolist()
    live = [i for i, n in enumerate(slots) if n >= 0]
    if c["type"] == Q8_0:
        out = []
        for x in (k, v):
            x = x.float().double().reshape(t, kv, d // 32, 32)  # a block is made of the 32-bit values
            step = (x.abs().max(-1, keepdim=True).values.float() / 127).half().double()
            y = torch.zeros_like(x)
            y[live] = (torch.where(step > 0, (x / step).round(), 0).clamp(-127, 127) * step)[live]
            out.append(y.reshape(t, kv * d))
        return q.reshape(t, -1), out[0], out[1]
    ks = torch.zeros(s["pages"] * page, kv, d, dtype=torch.float64, device="cuda")
    vs = torch.zeros_like(ks)
    to = [slots[i] for i in live]
    ks[to], vs[to] = k[live], v[live]
    ks = ks.view(s["pages"], page, kv, d).transpose(1, 2).reshape(s["pages"], -1)
    vs = vs.view(s["pages"], page // 16, 16, kv, d).permute(0, 3, 1, 4, 2).reshape(s["pages"], -1)
    return q.reshape(t, -1), ks, vs


def _exact_attn(s):
    c = s["case"]
    h, kv, d, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(s["rows"], kv, h // kv, d, dtype=torch.float64, device="cuda")
    start = s["start"].tolist()
    for b, n in enumerate(s["ctx"].tolist()):
        k, v = (x[0, :, :n] for x in _pages(s, s["table"][b:b + 1, :-(-n // page)]))
        new = start[b + 1] - start[b]
        for i in range(kv):
            k64, v64 = k[i].double(), v[i].double()
            for j in range(new):
                last = n - new + j
                first = max(0, last - c["window"] + 1) if c["window"] else 0
                q = s["q"][start[b] + j].view(kv, h // kv, d)[i].double()
                w = torch.softmax(q @ k64[first:last + 1].t() * d ** -0.5, -1)
                out[start[b] + j, i] = w @ v64[first:last + 1]
    return out.reshape(s["rows"], h * d)
