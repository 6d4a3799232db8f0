"""GPU: the paged key-value cache operators (include/kqkv.h) against kv_ref,
plain numpy in 64 bits.

Tolerances.  The plan is whole numbers.  A rotated value is computed in 64 bits
and rounded once: half a step, 2^-24 of the value, plus an angle error of pos
* 2^-51 times the pair's size (and the fp16 cache's half step, 2^-11, or 2^-25
below the normal range).  Q8_0 blocks are compared with the blocks of the
library's own rotated values.  The attention's bound is derived at
kv_ref.attn."""
import numpy as np
import pytest

import kqsynth
import kv_ref
import oracle

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu

F16, Q8 = kq.KQKV_F16, kq.KQKV_Q8_0


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(v):
    return dev(np.asarray(v, dtype=np.int32))


def zeros(*n):
    return torch.zeros(*n, dtype=torch.int32, device="cuda")


# ---- plan -----------------------------------------------------------------------

def plan_state(rng, B, page, stride, n_pages, max_ctx, extra=0):
    """Requests of random lengths holding shuffled pages (some more than they
    need), and the rest of the pages on the free list."""
    ctx = rng.integers(0, max_ctx + 1, B).astype(np.int32)
    held = (-(-ctx // page) + rng.integers(0, extra + 1, B)).astype(np.int32)
    held = np.minimum(held, stride).astype(np.int32)
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((B, stride), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(n_pages, -9, np.int32)
    free[:n_pages - at] = ids[at:]
    return ctx, held, table, free, n_pages - at


def run_plan(ctx, new, page, table, held, free, n_free, T, in_place=False):
    B, stride = table.shape
    d = dict(ctx=i32(ctx), new=i32(new), table=i32(table), held=i32(held), free=i32(free), n=i32([n_free]))
    out = (dict(held=d["held"], n=d["n"], ctx=d["ctx"]) if in_place else
           dict(held=zeros(B) - 5, n=zeros(1) - 5, ctx=zeros(B) - 5))
    slots, pos, start, err = zeros(T) - 3, zeros(T) - 3, zeros(B + 1) - 3, zeros(1)
    for _ in range(1 if in_place else 2):      # a repeated call gives the same
        kq.kqkv_plan(B, d["ctx"], d["new"], page, d["table"], stride, d["held"], out["held"], d["free"], len(free), d["n"],
                     out["n"], T, slots, pos, start, out["ctx"], err)
    torch.cuda.synchronize()
    c = lambda t: t.cpu().numpy()  # noqa: E731
    return dict(table=c(d["table"]), held=c(out["held"]), free=c(d["free"]), n_free=int(out["n"]), slots=c(slots), pos=c(pos),
                start=c(start), ctx=c(out["ctx"]), err=int(err))


def same_plan(got, want):
    for k in want:
        assert np.array_equal(got[k], want[k]), k


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,max_ctx,most", [(1, 16, 0, 1), (1, 16, 100, 1), (3, 48, 50, 8), (17, 16, 300, 1),
                                                 (64, 32, 1000, 200), (1000, 64, 200, 3), (1024, 16, 40, 5),
                                                 (1025, 16, 40, 1), (2500, 32, 100, 9), (5000, 16, 20, 2)])
def test_plan(B, page, max_ctx, most, in_place):
    rng = np.random.default_rng(B + most)
    stride = -(-(max_ctx + most) // page) + 2
    ctx, held, table, free, n_free = plan_state(rng, B, page, stride, B * stride + 3, max_ctx, 1)
    new = rng.integers(-1, most + 1, B).astype(np.int32)
    T = int(np.maximum(new, 0).sum()) + int(rng.integers(0, 20))
    want = kv_ref.plan(ctx, new, page, table, held, free, len(free), n_free, T)
    assert not want["err"]
    same_plan(run_plan(ctx, new, page, table, held, free, n_free, T, in_place), want)


def test_plan_takes_the_pages_just_given_back():
    # nothing is free but what two requests give back in the same step
    page, stride = 16, 4
    ctx, held = np.array([40, 5, 64, 0], np.int32), np.array([3, 1, 4, 0], np.int32)
    table = np.array([[9, 1, 5, -1], [3, -1, -1, -1], [0, 2, 4, 6], [-1, -1, -1, -1]], np.int32)
    new = np.array([-1, 30, -1, 64], np.int32)
    free = np.full(10, -1, np.int32)
    want = kv_ref.plan(ctx, new, page, table, held, free, 10, 0, 100)
    assert not want["err"] and want["n_free"] == 1
    same_plan(run_plan(ctx, new, page, table, held, free, 0, 100), want)
    same_plan(run_plan(ctx, new, page, table, held, free, 0, 100, in_place=True), want)


@pytest.mark.parametrize("case", ["pages", "table", "rows", "ctx", "held", "held_far", "n_free", "n_free_far", "overflow"])
@pytest.mark.parametrize("B", [5, 1500])
def test_plan_all_or_nothing(case, B):
    rng = np.random.default_rng(5)
    page, stride = 16, 8
    ctx, held, table, free, n_free = plan_state(rng, B, page, stride, B * stride, 60)
    new = np.ones(B, np.int32)
    new[1] = -1
    T = B
    at = B - 1
    if case == "pages":
        n_free, new[:] = 1, 20
        T = 20 * B
    elif case == "table":
        new[at] = stride * page
        T = B + stride * page
    elif case == "rows":
        T = B - 3
    elif case == "ctx":
        ctx[at] = -1
    elif case == "held":
        held[at] = -1
    elif case == "held_far":
        held[at] = stride + 1
    elif case == "n_free":
        n_free = -1
    elif case == "n_free_far":
        n_free = len(free) + 1
    elif case == "overflow":
        ctx[at] = new[at] = 2 ** 31 - 1
    want = kv_ref.plan(ctx, new, page, table, held, free, len(free), n_free, T)
    assert want["err"] == 1 and (want["slots"] == -1).all()
    same_plan(run_plan(ctx, new, page, table, held, free, n_free, T), want)
    same_plan(run_plan(ctx, new, page, table, held, free, n_free, T, in_place=True), want)


def test_plan_of_a_bad_page_and_no_rows():
    table, free = np.array([[99, -1, 0]], np.int32), np.arange(3, dtype=np.int32)
    got = run_plan([14], [4], 16, table, [1], free, 2, 4)
    want = kv_ref.plan(np.array([14], np.int32), np.array([4], np.int32), 16, table, np.array([1], np.int32), free, 3, 2, 4)
    same_plan(got, want)
    assert list(got["slots"]) == [-1, -1, 16, 17]
    # only requests that end or wait: no rows, slots and pos may be NULL
    d = [i32(v) for v in ([20, 3], [-1, 0])]
    t, held, f, n, start = i32([[2, 1], [0, -1]]), i32([2, 1]), i32([-1, -1, -1]), i32([0]), zeros(3)
    kq.kqkv_plan(2, d[0], d[1], 16, t, 2, held, held, f, 3, n, n, 0, None, None, start, d[0], None)
    assert d[0].tolist() == [0, 3] and held.tolist() == [0, 1] and f.tolist() == [2, 1, -1] and n.item() == 2


def test_plan_keeps_the_pages_of_rejected_tokens():
    # a verify pass of 8 over a page's end, 6 rejected, the next step of 8
    page, free = 16, np.arange(10, dtype=np.int32)
    table = np.full((1, 4), -1, np.int32)
    table[0, 0] = 7
    ctx, held, n, tab, fr = i32([12]), i32([1]), i32([7]), i32(table), i32(free)
    slots, pos, start, err = zeros(8), zeros(8), zeros(2), zeros(1)
    step = lambda new: kq.kqkv_plan(1, ctx, i32([new]), page, tab, 4, held, held, fr, 10, n, n, 8, slots, pos, start, ctx, err)  # noqa: E731
    step(8)
    first = slots.tolist()
    assert held.item() == 2 and n.item() == 6 and ctx.item() == 20
    ctx.fill_(14)
    step(8)
    assert held.item() == 2 and n.item() == 6 and ctx.item() == 22 and err.item() == 0
    assert slots.tolist()[:6] == first[2:] and pos.tolist() == list(range(14, 22))


# ---- rotary positions and store ---------------------------------------------------

def store_inputs(rng, T, q_heads, kv_heads, dim, page, axes, far, fused, gap=0):
    w = (q_heads + 2 * kv_heads) * dim
    if fused:
        x = dev(rng.standard_normal((T, w + gap)).astype(np.float32))
        q, k, v = x[:, :q_heads * dim], x[:, q_heads * dim:(q_heads + kv_heads) * dim], x[:, (q_heads + kv_heads) * dim:w]
    else:
        q, k, v = (dev(rng.standard_normal((T, n * dim)).astype(np.float32)) for n in (q_heads, kv_heads, kv_heads))
    n_pages = -(-T // page) + 3
    slots = rng.permutation(n_pages * page)[:T] if rng.random() < 0.5 else np.arange(5, 5 + T)
    slots = slots.astype(np.int32)
    slots[rng.random(T) < 0.1] = -1
    pos = rng.integers(0, far, (axes, T)).astype(np.int32)
    return q, k, v, slots, pos, n_pages


def device_cache(c):
    k, v = dev(c.k), dev(c.v)
    return kq.KVCache(c.type, c.heads, c.dim, c.page, c.n_pages, k, v), k, v


@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("T,q_heads,kv_heads,dim,page,style,rot,sections,far,fused", [
    (1, 32, 8, 128, 16, 0, 128, None, 10000, False),
    (1, 1, 1, 32, 16, 1, 2, None, 2 ** 31 - 1, False),
    (7, 8, 2, 64, 48, 1, 64, None, 100, True),
    (33, 5, 5, 96, 32, 0, 96, [16, 16, 16], 5000, True),
    (16, 64, 8, 128, 64, 0, 128, [16, 24, 24], 100000, False),
    (19, 12, 1, 256, 16, 1, 128, [64, 0, 0, 0], 3000000, False),
    (300, 3, 3, 160, 16, 0, 40, [0, 5, 15], 1000, True),
    (65, 71, 1, 64, 128, 0, 64, None, 2000, False),
    (2, 0, 4, 224, 256, 1, 224, None, 2000, False),
    (129, 6, 2, 192, 16, 0, 190, None, 2000, True),
])
def test_rope_store(type, T, q_heads, kv_heads, dim, page, style, rot, sections, far, fused):
    rng = np.random.default_rng(T + dim)
    sections = sections or [rot // 2]
    q, k, v, slots, pos, n_pages = store_inputs(rng, T, q_heads, kv_heads, dim, page, len(sections), far, fused, 4)
    factors = (1 + rng.random(rot // 2)).astype(np.float32) if T % 2 else None
    ref = kv_ref.Cache(type, kv_heads, dim, page, n_pages)
    cache, kb, vb = device_cache(ref)
    fd = dev(factors) if factors is not None else None
    rope = kq.KVRope(style, rot, 500000.0, sections, fd)
    gap = 8
    q_out = torch.full((T, q_heads * dim + gap), 7.0, device="cuda")
    kq.kqkv_rope_store(cache, rope, T, dev(pos), T, dev(slots), q_heads, q if q_heads else None, q.stride(0) if q_heads else 0,
                       q_out if q_heads else None, q_out.stride(0), k, k.stride(0), v, v.stride(0))
    torch.cuda.synchronize()
    kn, vn, qn = k.cpu().numpy().reshape(T, kv_heads, dim), v.cpu().numpy().reshape(T, kv_heads, dim), q.cpu().numpy()
    size = lambda x: np.hypot(*[np.abs(x).max()] * 2)  # noqa: E731
    angle = float(pos.max()) * 2.0 ** -51
    if q_heads:
        want = kv_ref.rope(qn.reshape(T, q_heads, dim), pos, style, rot, 500000.0, sections, factors).reshape(T, -1)
        got = q_out.cpu().numpy()
        assert (got[:, q_heads * dim:] == 7.0).all()
        err = np.abs(got[:, :q_heads * dim] - want)
        assert (err <= 2.0 ** -24 * np.abs(want) + (angle + 2.0 ** -48) * size(qn)).all()
    turned = kv_ref.rope(kn, pos, style, rot, 500000.0, sections, factors)
    # what was there before stays but at the slots
    if type == F16:
        for t in range(T):
            if slots[t] >= 0:
                ref.put(slots[t], np.zeros_like(kn[t]), vn[t])
        got = kv_ref.Cache(type, kv_heads, dim, page, n_pages)
        got.k, got.v = kb.cpu().numpy(), vb.cpu().numpy()
        assert np.array_equal(got.v, ref.v)
        for t in range(T):
            if slots[t] < 0:
                continue
            w = turned[t]
            e = np.abs(got.get(slots[t])[0] - w)
            assert (e <= np.maximum(2.0 ** -11 * (1 + 2.0 ** -12) * np.abs(w), 2.0 ** -25) + (angle + 2.0 ** -23) * size(kn)).all(), t
            got.put(slots[t], np.zeros_like(kn[t]), vn[t])
        assert np.array_equal(got.k, ref.k)
    else:
        # the library's own fp32 rotation of k (its q path), so that no quant sits on another side of a border
        kr = torch.empty(T, kv_heads * dim, device="cuda")
        kq.kqkv_rope_store(cache, rope, T, dev(pos), T, None, kv_heads, k, k.stride(0), kr, kv_heads * dim, None, 0, None, 0)
        kr = kr.cpu().numpy().reshape(T, kv_heads, dim)
        assert (np.abs(kr - turned) <= 2.0 ** -24 * np.abs(turned) + (angle + 2.0 ** -48) * size(kn)).all()
        for t in range(T):
            if slots[t] >= 0:
                ref.put(slots[t], kr[t], vn[t])
        assert np.array_equal(kb.cpu().numpy(), ref.k)
        assert np.array_equal(vb.cpu().numpy(), ref.v)


@pytest.mark.parametrize("type", [F16, Q8])
def test_binding_refuses_short_buffers(type):
    n = kq.kqkv_page_bytes(type, 2, 64, 16)
    t = torch.zeros(3 * n, dtype=torch.uint8, device="cuda")
    kq.KVCache(type, 2, 64, 16, 3, t, t)
    for k, v in ((t[:-1], t), (t, t[:-1]), (torch.zeros(3 * n, 2, dtype=torch.uint8, device="cuda")[:, 0], t)):
        with pytest.raises(ValueError):
            kq.KVCache(type, 2, 64, 16, 3, k, v)


def test_scales_between_two_halves():
    # largest magnitudes whose 127th rounds to one half as a product with the reciprocal and to the next as a quotient
    rng = np.random.default_rng(31)
    top = np.array([0x3FFF9CC1, 0x3FFE1FC1], dtype=np.uint32).view(np.float32)
    assert ((top * (np.float32(1) / np.float32(127))).astype(np.float16) != (top / np.float32(127)).astype(np.float16)).all()
    T, H, D, page = 32, 4, 32, 16
    m = rng.choice(np.concatenate([top, -top]), (2, T, H))
    x = (rng.uniform(-0.9, 0.9, (2, T, H, D)) * m[..., None]).astype(np.float32)
    x[0, :, :, 7], x[1, :, :, 19] = m
    ref = kv_ref.Cache(Q8, H, D, page, 2)
    cache, kb, vb = device_cache(ref)
    kq.kqkv_rope_store(cache, None, T, None, 0, i32(np.arange(T)), 0, None, 0, None, 0, dev(x[0].reshape(T, -1)), H * D,
                       dev(x[1].reshape(T, -1)), H * D)
    for t in range(T):
        ref.put(t, x[0, t], x[1, t])
    assert np.array_equal(kb.cpu().numpy().reshape(-1), ref.k.reshape(-1))
    assert np.array_equal(vb.cpu().numpy().reshape(-1), ref.v.reshape(-1))


@pytest.mark.parametrize("type", [F16, Q8])
def test_store_without_rotation_in_place_and_load(type):
    rng = np.random.default_rng(9)
    T, H, D, page, n = 37, 3, 96, 32, 4
    k, v = (rng.standard_normal((T, H, D)).astype(np.float32) * 10.0 ** rng.integers(-6, 4, (T, 1, 1)) for _ in range(2))
    k, v = k.astype(np.float32), v.astype(np.float32)
    k[3] = 0                                   # a scale of 0
    k[4, 1, 5], k[5, 2, 40], v[6, 0, 95] = np.inf, np.nan, -np.inf
    k[7] *= np.float32(1e-12)                  # the scale underflows
    v[8, 0, :32] = np.float32(1e30)            # past every fp16 scale
    slots = rng.permutation(n * page)[:T].astype(np.int32)
    slots[[0, 11, 20]] = [-1, n * page, -2 ** 31]
    ref = kv_ref.Cache(type, H, D, page, n)
    cache, kb, vb = device_cache(ref)
    kq.kqkv_rope_store(cache, None, T, None, 0, dev(slots), 0, None, 0, None, 0, dev(k.reshape(T, -1)), H * D, dev(v.reshape(T, -1)), H * D)
    ok = [t for t in range(T) if 0 <= slots[t] < n * page]
    for t in ok:
        ref.put(slots[t], k[t], v[t])
    got = kv_ref.Cache(type, H, D, page, n)
    got.k, got.v = kb.cpu().numpy(), vb.cpu().numpy()
    ko, vo = (torch.full((T, H * D), 5.0, device="cuda") for _ in range(2))
    kq.kqkv_load(cache, T, dev(slots), ko, vo)
    ko, vo = ko.cpu().numpy(), vo.cpu().numpy()
    for t in range(T):
        if t not in ok:
            assert (ko[t] == 5).all() and (vo[t] == 5).all()
            continue
        (a, b), (wa, wb) = got.get(slots[t]), ref.get(slots[t])
        assert np.array_equal(a, wa, equal_nan=True) and np.array_equal(b, wb, equal_nan=True), t
        assert np.array_equal(ko[t].reshape(H, D), wa.astype(np.float32), equal_nan=True)
        assert np.array_equal(vo[t].reshape(H, D), wb.astype(np.float32), equal_nan=True)
    only = torch.full((T, H * D), 5.0, device="cuda")
    kq.kqkv_load(cache, T, dev(slots), None, only)
    assert np.array_equal(only.cpu().numpy(), vo, equal_nan=True)
    # q rotated in place, nothing stored
    q = rng.standard_normal((T, 2 * D)).astype(np.float32)
    qd, pos = dev(q), rng.integers(0, 50, (1, T)).astype(np.int32)
    before = kb.clone()
    kq.kqkv_rope_store(cache, kq.KVRope(1, 64, 100.0), T, dev(pos), T, None, 2, qd, 2 * D, qd, 2 * D, None, 0, None, 0)
    want = kv_ref.rope(q.reshape(T, 2, D), pos, 1, 64, 100.0, [32]).reshape(T, -1)
    assert (np.abs(qd.cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -44).all()
    assert torch.equal(before, kb)


# ---- attention ----------------------------------------------------------------------

def attn_case(rng, type, q_heads, kv_heads, dim, page, ctx, new, spare=2):
    stride = max(1, -(-max(ctx) // page)) + spare
    n_pages = sum(-(-c // page) for c in ctx) + 3
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(ctx), stride), -1, np.int32)
    at = 0
    for b, c in enumerate(ctx):
        n = -(-c // page)
        table[b, :n] = ids[at:at + n]
        at += n
    ref = kv_ref.Cache(type, kv_heads, dim, page, n_pages)
    ref.fill(rng, table, ctx)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = rng.standard_normal((int(start[-1]) + 3, q_heads * dim)).astype(np.float32)
    return ref, table, start, q


def run_attn(ref, table, ctx, start, q, q_heads, scale, window, max_q, max_ctx=None, gap=0, err=None, T=None, dc=None):
    cache = dc or device_cache(ref)[0]
    T = q.shape[0] if T is None else T
    B, n = len(ctx), q_heads * ref.dim
    qd = torch.full((q.shape[0], n + gap), float("nan"), device="cuda")
    qd[:, :n] = dev(q)
    out = torch.full((q.shape[0], n + gap), 3.0, device="cuda")
    max_ctx = max_ctx or max(1, max(ctx))
    nb = kq.kqkv_attn_workspace_bytes(cache, B, max_q, max_ctx, q_heads)
    ws = torch.full((max(nb, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    args = (cache, B, max_q, max_ctx, i32(ctx), i32(start), i32(table), table.shape[1], q_heads, T, qd, n + gap, scale, window, out,
            n + gap, ws, nb, err)
    kq.kqkv_attn(*args)
    first = out.clone()
    kq.kqkv_attn(*args)
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int32), out.view(torch.int32))      # reruns give the same bits
    got = out.cpu().numpy()
    assert (got[:, n:] == 3.0).all()
    return got[:, :n]


def check_attn(got, want, tol):
    d = np.abs(got - want)
    worst = (d / np.maximum(tol, 1e-300))[tol > 0]
    print("attention: worst %.3g of the bound" % (worst.max() if worst.size else 0))
    assert (d <= tol).all()


CASES = [
    # q_heads, kv_heads, dim, page, contexts, new tokens, window
    (8, 8, 128, 16, [1], [1], 0),
    (8, 1, 128, 16, [1, 2, 15, 16, 17, 31, 32, 33], [1] * 8, 0),
    (32, 8, 128, 16, [37], [1], 0),
    (64, 8, 128, 64, [200, 1, 0, 129], [1, 1, 0, 1], 0),
    (64, 8, 128, 16, [300, 41], [8, 3], 0),
    (16, 16, 64, 16, [500, 77, 130], [1, 2, 1], 100),
    (4, 4, 32, 48, [97, 48], [4, 4], 1),
    (12, 2, 96, 32, [250, 33, 5], [1, 5, 2], 40),
    (10, 1, 160, 128, [300], [8], 0),
    (6, 2, 192, 16, [123, 64], [7, 1], 0),
    (7, 1, 224, 256, [270], [1], 17),
    (16, 2, 256, 16, [333, 20], [1, 8], 0),
    (71, 1, 64, 16, [90], [2], 0),
    (130, 1, 32, 16, [70], [8], 33),
    (2, 1, 64, 16, [1500, 700], [1, 1], 0),
]


@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("q_heads,kv_heads,dim,page,ctx,new,window", CASES)
def test_attn(type, q_heads, kv_heads, dim, page, ctx, new, window):
    rng = np.random.default_rng(sum(ctx) + dim)
    ref, table, start, q = attn_case(rng, type, q_heads, kv_heads, dim, page, ctx, new)
    scale = 1 / np.sqrt(dim)
    err = zeros(1)
    got = run_attn(ref, table, ctx, start, q, q_heads, scale, window, max(max(new), 1), gap=4, err=err)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, q_heads, float(np.float32(scale)), window, out=np.full_like(q, 3.0))
    check_attn(got, want, tol)
    assert err.item() == 0


@pytest.mark.parametrize("type", [F16, Q8])
def test_attn_long_contexts_are_split(type):
    rng = np.random.default_rng(77)
    ctx, new = [9001, 3, 4500], [1, 1, 2]
    ref, table, start, q = attn_case(rng, type, 4, 2, 64, 64, ctx, new)
    got = run_attn(ref, table, ctx, start, q, 4, 0.125, 0, 2)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, 4, 0.125, 0, out=np.full_like(q, 3.0))
    check_attn(got, want, tol)
    # a max_ctx that is too short changes nothing but the speed
    got = run_attn(ref, table, ctx, start, q, 4, 0.125, 0, 2, max_ctx=1)
    check_attn(got, want, tol)
    # a window that leaves whole stretches of the context out
    got = run_attn(ref, table, ctx, start, q, 4, 0.125, 700, 2)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, 4, 0.125, 700, out=np.full_like(q, 3.0))
    check_attn(got, want, tol)


@pytest.mark.parametrize("type", [F16, Q8])
def test_attn_far_scores(type):
    # scores that differ by hundreds, the largest at the end, first and in the middle; magnitudes of q from 1e-20 to 1e4
    rng = np.random.default_rng(5)
    ctx, new = [300, 300, 300], [1, 1, 1]
    ref, table, start, q = attn_case(rng, type, 4, 1, 64, 16, ctx, new)
    for b, i in enumerate((0, 150, 299)):
        ref.put(table[b, i // 16] * 16 + i % 16, 20 * q[b].reshape(4, 64)[:1], np.ones((1, 64)))
    q[1] *= 1e-20
    q[2, 64:128] *= 1e4
    got = run_attn(ref, table, ctx, start, q, 4, 0.125, 0, 1)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, 4, 0.125, 0, out=np.full_like(q, 3.0))
    check_attn(got, want, np.minimum(tol, 1e3))


def test_attn_rows_without_tokens():
    # a length of 0 or below, a length shorter than the new tokens: rows before the first token are 0; rows that are
    # no request's stay
    rng = np.random.default_rng(6)
    ctx, new = [2, 0, 40], [5, 2, 1]
    ref, table, start, q = attn_case(rng, F16, 4, 2, 32, 16, ctx, new)
    got = run_attn(ref, table, ctx, start, q, 4, 0.2, 0, 5)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, 4, float(np.float32(0.2)), 0, out=np.full_like(q, 3.0))
    check_attn(got, want, tol)
    assert (got[:3] == 0).all() and (got[5:7] == 0).all() and (got[8:] == 3).all()
    got = run_attn(ref, table, [2, -5, 40], start, q, 4, 0.2, 0, 5)
    check_attn(got, want, tol)
    # more rows than max_q: the first ones are computed
    got = run_attn(ref, table, ctx, start, q, 4, 0.2, 0, 4)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, 4, float(np.float32(0.2)), 0, max_q=4, out=np.full_like(q, 3.0))
    check_attn(got, want, tol)
    # rows past T are not touched
    got = run_attn(ref, table, ctx, start, q, 4, 0.2, 0, 5, T=4)
    want, tol = kv_ref.attn(ref, table, ctx, start, q[:4], 4, float(np.float32(0.2)), 0)
    check_attn(got[:4], want, tol)
    assert (got[4:] == 3).all()


@pytest.mark.parametrize("type", [F16, Q8])
def test_attn_bad_pages_take_their_tokens_out(type):
    rng = np.random.default_rng(8)
    ctx, new = [100, 75, 64], [1, 2, 1]
    ref, table, start, q = attn_case(rng, type, 8, 2, 64, 16, ctx, new)
    table[0, 2], table[0, 6], table[2, :] = ref.n_pages, -1, 2 ** 30
    err = zeros(1)
    got = run_attn(ref, table, ctx, start, q, 8, 0.125, 0, 2, err=err)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, 8, 0.125, 0, out=np.full_like(q, 3.0))
    check_attn(got, want, tol)
    assert err.item() == 1 and (got[start[2]] == 0).all()
    # a length past the table
    ref, table, start, q = attn_case(rng, type, 8, 2, 64, 16, [64], [1], spare=0)
    for far in (65, 100, 2 ** 31 - 1):
        err = zeros(1)
        got = run_attn(ref, table, [far], start, q, 8, 0.125, 0, 1, err=err, max_ctx=64)
        want, tol = kv_ref.attn(ref, table, [far], start, q, 8, 0.125, 0, out=np.full_like(q, 3.0))
        check_attn(got, want, tol)
        assert err.item() == 1


def test_attn_on_another_stream_and_two_at_once():
    rng = np.random.default_rng(12)
    ctx, new = [3000, 100], [1, 1]
    made = [attn_case(rng, t, 8, 2, 64, 16, ctx, new) for t in (F16, Q8)]
    streams = [torch.cuda.Stream() for _ in made]
    outs = []
    for (ref, table, start, q), s in zip(made, streams):
        cache = device_cache(ref)
        nb = kq.kqkv_attn_workspace_bytes(cache[0], 2, 1, 3000, 8)
        d = (i32(ctx), i32(start), i32(table), dev(q), torch.zeros_like(dev(q)), torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda"))
        outs.append((cache, nb, d))
    torch.cuda.synchronize()
    for rep in range(5):
        for (ref, table, start, q), s, (cache, nb, d) in zip(made, streams, outs):
            with torch.cuda.stream(s):
                kq.kqkv_attn(cache[0], 2, 1, 3000, d[0], d[1], d[2], table.shape[1], 8, q.shape[0], d[3], 512, 0.125, 0, d[4], 512, d[5], nb)
    torch.cuda.synchronize()
    for (ref, table, start, q), (cache, nb, d) in zip(made, outs):
        want, tol = kv_ref.attn(ref, table, ctx, start, q, 8, 0.125, 0)
        check_attn(d[4].cpu().numpy(), want, tol)


@pytest.mark.parametrize("type", [F16, Q8])
def test_attn_hint_of_a_huge_context(type):
    # max_ctx only sets how the work is split and how lines are read: the largest one, on ordinary and empty requests
    rng = np.random.default_rng(14)
    ctx, new = [2500, 0, 31, 700], [1, 1, 0, 1]
    for q_heads, kv_heads, dim in ((8, 2, 128), (6, 3, 96), (4, 4, 32)):
        ref, table, start, q = attn_case(rng, type, q_heads, kv_heads, dim, 32, ctx, new)
        got = run_attn(ref, table, ctx, start, q, q_heads, dim ** -0.5, 0, 1, max_ctx=2 ** 31 - 1)
        want, tol = kv_ref.attn(ref, table, ctx, start, q, q_heads, float(np.float32(dim ** -0.5)), 0, out=np.full_like(q, 3.0))
        check_attn(got, want, tol)


@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("q_heads,dim,ctx,new,window", [(16, 64, [3000, 500], [8, 8], 0), (40, 32, [1700], [8], 900),
                                                         (24, 128, [1200, 40], [2, 1], 0), (5, 256, [1100], [7], 0)])
def test_attn_many_rows_over_cut_contexts(type, q_heads, dim, ctx, new, window):
    rng = np.random.default_rng(q_heads)
    ref, table, start, q = attn_case(rng, type, q_heads, 1, dim, 16, ctx, new)
    got = run_attn(ref, table, ctx, start, q, q_heads, dim ** -0.5, window, 8)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, q_heads, float(np.float32(dim ** -0.5)), window, out=np.full_like(q, 3.0))
    check_attn(got, want, tol)


@pytest.mark.parametrize("B,longest", [(65, 1500), (200, 90), (1000, 20)])
def test_attn_many_requests(B, longest):
    # more requests than a wave's lanes: lengths and rows are found over several rounds
    rng = np.random.default_rng(B)
    ctx = [int(n) for n in rng.integers(0, 40, B)]
    ctx[B // 2], ctx[-1] = longest, longest // 2
    new = [int(n) for n in rng.integers(0, 2, B)]
    new[B // 2] = new[-1] = 1
    ref, table, start, q = attn_case(rng, F16, 2, 1, 32, 16, ctx, new)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, 2, float(np.float32(0.18)), 0, out=np.full_like(q, 3.0))
    for max_ctx in (longest, 2 ** 31 - 1, 1):
        check_attn(run_attn(ref, table, ctx, start, q, 2, 0.18, 0, 1, max_ctx=max_ctx), want, tol)


@pytest.mark.parametrize("lengths", ["equal", "ragged", "one", "two_long"])
@pytest.mark.parametrize("type,B,heads", [(F16, 20, 8), (Q8, 40, 8), (F16, 64, 4), (Q8, 2, 8)])
def test_attn_cut_to_fill_the_device(type, B, heads, lengths):
    # fewer pieces than the lengths would take: their size is searched for
    rng = np.random.default_rng(B + heads)
    most = 1700
    ctx = {"equal": [most] * B, "ragged": [int(n) for n in rng.integers(0, most, B)], "one": [0] * (B - 1) + [most],
           "two_long": [most, most - 33] + [int(n) for n in rng.integers(0, 40, B - 2)]}[lengths]
    new = [1 if n else 0 for n in ctx]
    ref, table, start, q = attn_case(rng, type, heads, heads, 32, 64, ctx, new)
    want, tol = kv_ref.attn(ref, table, ctx, start, q, heads, float(np.float32(0.18)), 0, out=np.full_like(q, 3.0))
    for max_ctx in (most, 10 ** 6):
        check_attn(run_attn(ref, table, ctx, start, q, heads, 0.18, 0, 1, max_ctx=max_ctx), want, tol)


@pytest.mark.parametrize("type", [F16, Q8])
def test_pages_past_four_gibibytes(type):
    # the last pages of a cache of over 4 GiB, K and V each: written, read back and attended to
    rng = np.random.default_rng(4)
    H, D, page, n = 8, 256, 64, 70
    pb = kq.kqkv_page_bytes(type, H, D, page)
    n_pages = (1 << 32) // pb + 9
    kb, vb = (torch.empty(n_pages * pb, dtype=torch.uint8, device="cuda") for _ in range(2))
    cache = kq.KVCache(type, H, D, page, n_pages, kb, vb)
    k, v = (rng.standard_normal((n, H, D)).astype(np.float32) for _ in range(2))
    far = np.array([[n_pages - 1, n_pages - 2]], np.int32)
    slots = far[0][np.arange(n) // page] * page + np.arange(n) % page
    kq.kqkv_rope_store(cache, None, n, None, 0, i32(slots), 0, None, 0, None, 0, dev(k.reshape(n, -1)), H * D, dev(v.reshape(n, -1)), H * D)
    small = kv_ref.Cache(type, H, D, page, 2)
    for t in range(n):
        small.put(t, k[t], v[t])
    ko, vo = (torch.zeros(n, H * D, device="cuda") for _ in range(2))
    kq.kqkv_load(cache, n, i32(slots), ko, vo)
    want = [small.get(t) for t in range(n)]
    assert np.array_equal(ko.cpu().numpy().reshape(n, H, D), np.stack([a for a, _ in want]).astype(np.float32))
    assert np.array_equal(vo.cpu().numpy().reshape(n, H, D), np.stack([a for _, a in want]).astype(np.float32))
    q = rng.standard_normal((1, H * D)).astype(np.float32)
    got = run_attn(small, far, [n], [0, 1], q, H, 0.0625, 0, 1, dc=cache)
    want, tol = kv_ref.attn(small, np.array([[0, 1]]), [n], [0, 1], q, H, 0.0625, 0)
    check_attn(got, want, tol)


def test_attn_two_graphs_share_a_workspace():
    # captured with different sizes, replayed in turn on one stream with eager work between
    rng = np.random.default_rng(15)
    made = []
    for ctx, new, heads, type in (([1900, 30], [1, 1], 8, F16), ([700, 600, 5], [4, 1, 2], 4, Q8)):
        ref, table, start, q = attn_case(rng, type, heads, 2, 64, 16, ctx, new)
        cache = device_cache(ref)
        nb = kq.kqkv_attn_workspace_bytes(cache[0], len(ctx), 4, 2000, heads)
        made.append((ref, table, start, q, ctx, heads, cache, nb, (i32(ctx), i32(start), i32(table), dev(q), torch.zeros(q.shape, device="cuda"))))
    ws = torch.full((max(m[7] for m in made),), 0xFF, dtype=torch.uint8, device="cuda")
    graphs = []
    torch.cuda.synchronize()
    for ref, table, start, q, ctx, heads, cache, nb, d in made:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            kq.kqkv_attn(cache[0], len(ctx), 4, 2000, d[0], d[1], d[2], table.shape[1], heads, q.shape[0], d[3], q.shape[1], 0.125, 0,
                         d[4], q.shape[1], ws, nb)
        graphs.append(g)
    wants = [kv_ref.attn(m[0], m[1], m[4], m[2], m[3], m[5], 0.125, 0) for m in made]
    for rep in range(4):
        for i in (0, 1, 1, 0):
            made[i][8][4].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            check_attn(made[i][8][4].cpu().numpy(), *wants[i])
            torch.empty(1 << 20, device="cuda").normal_()


# ---- together --------------------------------------------------------------------------

def test_steps_of_a_layer_between_the_projections():
    """Decode and verify steps of three requests through a layer's attention: q, k and v by one grouped call, the plan,
    rotary positions and store, the attention, the output projection; requests come, go and take tokens back."""
    rng = np.random.default_rng(21)
    hidden, q_heads, kv_heads, dim, page = 256, 4, 2, 64, 16
    types = [kq.KQ_TYPE_Q4_K, kq.KQ_TYPE_Q4_K, kq.KQ_TYPE_Q6_K, kq.KQ_TYPE_Q8_0]
    shapes = [(q_heads * dim, hidden), (kv_heads * dim, hidden), (kv_heads * dim, hidden), (hidden, q_heads * dim)]
    W = [kqsynth.matrix(t, n, k, kqsynth.rng_for(50, i)) for i, (t, (n, k)) in enumerate(zip(types, shapes))]
    dense = [oracle.dequant(t, w, n * k).reshape(n, k).astype(np.float64) for t, w, (n, k) in zip(types, W, shapes)]
    Wd = [dev(w.reshape(-1)) for w in W]
    B, stride, n_pages = 3, 6, 14
    for type in (F16, Q8):
        ref = kv_ref.Cache(type, kv_heads, dim, page, n_pages)
        cache, kb, vb = device_cache(ref)
        rope = kq.KVRope(kq.KQKV_ROPE_PAIRS, dim, 10000.0)
        ctx, held, table, n_free, free = zeros(B), zeros(B), zeros(B, stride) - 1, i32([n_pages]), i32(np.arange(n_pages))
        start, err = zeros(B + 1), zeros(1)
        nb = kq.kqkv_attn_workspace_bytes(cache, B, 8, stride * page, q_heads)
        ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
        tokens = [[] for _ in range(B)]                       # each request's stored (k, v), exact cache values
        for step, new in enumerate([[5, 1, 0], [1, 8, 2], [8, 1, 1], [-1, 7, 4], [8, 0, -1], [1, 3, 6], [4, 3, 1]]):
            T = sum(max(n, 0) for n in new)
            x = rng.standard_normal((T, hidden)).astype(np.float32)
            xd = dev(x)
            q, k, v, o, y = (torch.zeros(T, n, device="cuda") for n in (q_heads * dim, kv_heads * dim, kv_heads * dim, q_heads * dim, hidden))
            slots, pos = zeros(T), zeros(T)
            kq.kqkv_plan(B, ctx, i32(new), page, table, stride, held, held, free, n_pages, n_free, n_free, T, slots, pos, start, ctx, err)
            for r in range(0, T, 8):                            # the projections take up to 8 rows
                m = min(8, T - r)
                kq.kq_qgemv_multi(types[:3], Wd[:3], [s[0] for s in shapes[:3]], hidden, xd[r:], m, [q[r:], k[r:], v[r:]])
            kq.kqkv_rope_store(cache, rope, T, pos, T, slots, q_heads, q, q_heads * dim, q, q_heads * dim, k, kv_heads * dim, v, kv_heads * dim)
            kq.kqkv_attn(cache, B, 8, stride * page, ctx, start, table, stride, q_heads, T, q, q_heads * dim, dim ** -0.5, 0, o, q_heads * dim, ws, nb, err)
            for r in range(0, T, 8):
                kq.kq_qgemv(types[3], Wd[3], hidden, q_heads * dim, o[r:], min(8, T - r), y[r:])
            torch.cuda.synchronize()
            assert err.item() == 0
            # the same from the dense weights; the cache values from a dense rotation, rounded as the cache holds them
            st, p0, sl = start.tolist(), pos.tolist(), slots.tolist()
            for b in range(B):
                if new[b] < 0:
                    tokens[b] = []
            wk = kv_ref.rope((x @ dense[1].T).reshape(T, kv_heads, dim), [p0], 1, dim, 1e4, [dim // 2])
            wq = kv_ref.rope((x @ dense[0].T).reshape(T, q_heads, dim), [p0], 1, dim, 1e4, [dim // 2])
            wv = (x @ dense[2].T).reshape(T, kv_heads, dim)
            got = kv_ref.Cache(type, kv_heads, dim, page, n_pages)
            got.k, got.v = kb.cpu().numpy(), vb.cpu().numpy()
            for b in range(B):
                for j, t in enumerate(range(st[b], st[b + 1])):
                    assert p0[t] == len(tokens[b])
                    gk, gv = got.get(sl[t])
                    step_k = np.abs(wk[t]).max() / 127 if type == Q8 else np.abs(wk[t]).max() * 2.0 ** -11
                    step_v = np.abs(wv[t]).max() / 127 if type == Q8 else np.abs(wv[t]).max() * 2.0 ** -11
                    assert np.abs(gk - wk[t]).max() <= step_k and np.abs(gv - wv[t]).max() <= step_v
                    tokens[b].append((gk, gv))
                n = len(tokens[b])
                assert n == ctx[b].item()
                for j, t in enumerate(range(st[b], st[b + 1])):
                    ks = np.stack([a for a, _ in tokens[b][:p0[t] + 1]])
                    vs = np.stack([a for _, a in tokens[b][:p0[t] + 1]])
                    out = np.zeros((q_heads, dim))
                    for h in range(q_heads):
                        s = ks[:, h // 2] @ wq[t, h] * dim ** -0.5
                        w = np.exp(s - s.max())
                        out[h] = w @ vs[:, h // 2] / w.sum()
                    want = dense[3] @ out.reshape(-1)
                    # scores within 1e-4 of their size (the projections' bound) and the output projection's bound
                    A = np.abs(ks).max() * np.abs(wq[t]).sum(-1).max() * dim ** -0.5
                    tol = (np.abs(dense[3]) @ np.full(q_heads * dim, np.abs(vs).max())) * (4e-4 * A + 4e-4) + 1e-6
                    assert (np.abs(y[t].cpu().numpy() - want) <= tol).all(), (step, b, j)
            # the verify pass keeps some of its tokens
            if step == 2:
                ctx[0] -= 5
                tokens[0] = tokens[0][:-5]


def test_captured_steps_follow_the_lengths():
    """plan, rotation and store, and attention captured once and replayed over steps, against the same calls made eagerly."""
    rng = np.random.default_rng(31)
    B, q_heads, kv_heads, dim, page, stride, n_pages, T = 4, 8, 2, 64, 16, 40, 160, 8
    xs = [[dev(rng.standard_normal((T, n * dim)).astype(np.float32)) for n in (q_heads, kv_heads, kv_heads)] for _ in range(6)]
    news = [i32(n) for n in ([1, 2, 3, 1], [1, 1, 1, 1], [8, 0, 0, 0], [0, 0, -1, 5], [2, 2, 2, 2], [1, 1, 0, 1])]
    sides = []
    for side in range(2):
        kb, vb = (torch.zeros(n_pages, kq.kqkv_page_bytes(Q8, kv_heads, dim, page), dtype=torch.uint8, device="cuda") for _ in range(2))
        d = dict(cache=kq.KVCache(Q8, kv_heads, dim, page, n_pages, kb, vb), rope=kq.KVRope(0, dim, 1e4), ctx=i32([500, 3, 17, 250]),
                 held=zeros(B), table=zeros(B, stride) - 1, free=i32(np.arange(n_pages)), n=i32([n_pages]), new=zeros(B), start=zeros(B + 1),
                 slots=zeros(T), pos=zeros(T), err=zeros(1), x=[torch.empty_like(a) for a in xs[0]], out=torch.zeros(T, q_heads * dim, device="cuda"))
        nb = kq.kqkv_attn_workspace_bytes(d["cache"], B, 8, stride * page, q_heads)
        d["ws"], d["nb"] = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda"), nb
        sides.append(d)

    def step(d):
        kq.kqkv_plan(B, d["ctx"], d["new"], page, d["table"], stride, d["held"], d["held"], d["free"], n_pages, d["n"], d["n"], T,
                     d["slots"], d["pos"], d["start"], d["ctx"], d["err"])
        q, k, v = d["x"]
        kq.kqkv_rope_store(d["cache"], d["rope"], T, d["pos"], T, d["slots"], q_heads, q, q_heads * dim, q, q_heads * dim, k, kv_heads * dim, v, kv_heads * dim)
        kq.kqkv_attn(d["cache"], B, 8, stride * page, d["ctx"], d["start"], d["table"], stride, q_heads, T, q, q_heads * dim, 0.125, 0,
                     d["out"], q_heads * dim, d["ws"], d["nb"], d["err"])

    eager, graphed = sides
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step(graphed)
    for n, x in zip(news, xs):
        for d in sides:
            d["new"].copy_(n)
            for a, b in zip(d["x"], x):
                a.copy_(b)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("ctx", "held", "table", "free", "n", "slots", "pos", "start", "err", "out"):
            assert torch.equal(eager[k], graphed[k]), k
        torch.empty(1 << 20, device="cuda").normal_()
    assert eager["err"].item() == 0
