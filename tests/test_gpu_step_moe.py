"""GPU: kqstep_moe against 64 bits: every block format in both places, routing
rules, ties, sizes, strides, in place, captured graphs."""
import itertools

import numpy as np
import pytest

import kqsynth
import step_ref
from kqsynth import Q2_K, Q3_K, Q4_0, Q4_K, Q5_K, Q6_K, Q8_0

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def device_layer(c):
    return kq.MoELayer(c["E"], c["k"], c["hidden"], c["inner"], c["gate_type"], dev(c["gate"]), dev(c["up"]), c["down_type"], dev(c["down"]),
                       dev(c["router"]), dev(c["bias"]), c["score"], c["renorm"], c["scale"], c["act"])


def call(c, x, add=None, layer=None, y=None, ids=True):
    layer = layer or device_layer(c)
    T, H = x.shape
    n = kq.kqstep_moe_workspace_bytes(layer, T)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")          # NaN all over: scratch needs no preparation
    y = torch.full((T, H), float("nan"), device="cuda") if y is None else y
    out = (torch.full((T, c["k"]), -7, dtype=torch.int32, device="cuda"), torch.full((T, c["k"]), float("nan"), device="cuda")) if ids else (None, None)
    kq.kqstep_moe(layer, T, x, x.stride(0), add, add.stride(0) if add is not None else 0, y, y.stride(0), *out, ws, n)
    return y, out[0], out[1]


def check(c, x, add, got):
    y, ids, p = (g.cpu().numpy() for g in got)
    want, wids, wp, tol = step_ref.moe(c, x, add)
    assert np.array_equal(ids, wids), (ids, wids)
    # the weights are rounded once (64-bit exponentials and sums: below 2^-40)
    assert np.all(np.abs(p - wp) <= np.abs(wp) * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -149)
    err = np.abs(y - want)
    assert np.all(err <= tol), (err / tol).max()
    # and far below that bound as a whole: sums of fp32 roundings that fall either way, of terms whose quants' offsets make them up to
    # about four times as large as the weights; sqrt(roundings) * 2^-24 * 4 stays below 2^-16
    assert np.linalg.norm(err) <= 2.0 ** -16 * np.linalg.norm(want)
    return y


def case(seed, T, add=True, **kw):
    rng = np.random.default_rng(seed)
    c = step_ref.layer(rng, **kw)
    x = rng.standard_normal((T, kw["hidden"])).astype(np.float32)
    return c, x, rng.standard_normal(x.shape).astype(np.float32) if add else None


KINDS = [Q4_0, Q8_0, Q2_K, Q3_K, Q4_K, Q5_K, Q6_K]


@pytest.mark.parametrize("gate,down", list(zip(KINDS, KINDS[3:] + KINDS[:3])) + [(Q4_K, Q6_K)])
def test_formats(gate, down):
    for T, E, k, H, F in ((1, 8, 2, 512, 256), (3, 6, 3, 768, 512)):
        c, x, a = case([gate, down, T], T, E=E, k=k, hidden=H, inner=F, gate_type=gate, down_type=down)
        check(c, x, a, call(c, dev(x), dev(a)))


@pytest.mark.parametrize("score,renorm,bias,scale,act", [(0, True, False, 1.0, 0), (0, False, False, 1.0, 1), (0, True, True, 2.5, 0), (1, True, False, 1.0, 0),
                                                         (1, True, True, 2.5, 1), (1, False, True, -0.5, 0)])
def test_routing_rules(score, renorm, bias, scale, act):
    for T in (1, 5):
        c, x, a = case([score, renorm, bias, T], T, E=21, k=5, hidden=256, inner=256, gate_type=Q4_K, down_type=Q4_K, score=score, renorm=renorm,
                       bias=bias, scale=scale, act=act)
        check(c, x, a, call(c, dev(x), dev(a)))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (8, 1, 1), (2, 16, 16), (1, 17, 16), (8, 3, 2), (4, 64, 7), (2, 65, 8), (2, 130, 9), (1, 1024, 10), (3, 1000, 1),
                                   (1, 12, 11)])
def test_expert_counts(T, E, k):
    c, x, a = case([T, E, k], T, E=E, k=k, hidden=64, inner=32, gate_type=Q8_0, down_type=Q4_0)
    check(c, x, a, call(c, dev(x), dev(a)))


@pytest.mark.parametrize("H,F,gate,down", [(32, 32, Q8_0, Q8_0), (96, 160, Q4_0, Q8_0), (608, 1184, Q8_0, Q4_0), (1024, 2048, Q6_K, Q4_K), (2048, 768, Q4_K, Q6_K),
                                           (2304, 256, Q5_K, Q3_K), (4096, 512, Q4_K, Q8_0), (4352, 1280, Q2_K, Q6_K), (256, 4352, Q4_K, Q5_K),
                                           (5120, 768, Q3_K, Q2_K), (2080, 1056, Q4_0, Q4_0), (8448, 256, Q4_K, Q4_K)])
def test_sizes(H, F, gate, down):
    for T in (1, 2):
        c, x, a = case([H, F, T], T, add=T == 1, E=5, k=2, hidden=H, inner=F, gate_type=gate, down_type=down)
        check(c, x, a, call(c, dev(x), dev(a)))


@pytest.mark.parametrize("T", range(1, 9))
def test_tokens(T):
    """Every number of tokens; a token's results do not depend on the others."""
    c, x, a = case([T], 8, E=9, k=4, hidden=512, inner=512, gate_type=Q4_K, down_type=Q6_K)
    layer = device_layer(c)
    y, ids, p = call(c, dev(x[:T]), dev(a[:T]), layer)
    check(c, x[:T], a[:T], (y, ids, p))
    one, i1, p1 = call(c, dev(x[T - 1:T]), dev(a[T - 1:T]), layer)
    assert torch.equal(one[0], y[T - 1]) and torch.equal(i1[0], ids[T - 1]) and torch.equal(p1[0], p[T - 1])


@pytest.mark.parametrize("k, hidden, inner, down", [(4, 2304, 256, Q4_K), (8, 2304, 512, Q6_K), (2, 512, 1184, Q8_0)])
def test_results_are_the_same_in_calls_of_any_size(k, hidden, inner, down):
    """Bit by bit, also where calls of other sizes split their rows differently."""
    c, x, a = case([9, k], 8, E=9, k=k, hidden=hidden, inner=inner, gate_type=Q4_K, down_type=down)
    layer = device_layer(c)
    y, ids, p = call(c, dev(x), dev(a), layer)
    check(c, x, a, (y, ids, p))
    for T in range(1, 8):
        for t0 in (0, 8 - T):
            part = call(c, dev(x[t0:t0 + T]), dev(a[t0:t0 + T]), layer)
            for one, all_ in zip(part, (y, ids, p)):
                assert torch.equal(one, all_[t0:t0 + T]), (T, t0)


def test_tokens_that_choose_the_same_experts():
    c, x, a = case([77], 6, E=20, k=6, hidden=256, inner=256, gate_type=Q5_K, down_type=Q4_0)
    x[1:] = x[0]
    check(c, x, a, call(c, dev(x), dev(a)))


@pytest.mark.parametrize("bias", [False, True])
def test_ties_go_to_the_lower_expert(bias):
    c, x, a = case([5], 2, E=70, k=6, hidden=256, inner=256, gate_type=Q4_K, down_type=Q4_K, bias=bias)
    c["router"][:] = c["router"][3]                                        # every logit the same
    if bias:
        c["bias"][:] = 0.25
        c["bias"][40] = 0.5
    y, ids, p = call(c, dev(x), dev(a))
    assert ids.tolist() == [[40, 0, 1, 2, 3, 4] if bias else list(range(6))] * 2
    check(c, x, a, (y, ids, p))


@pytest.mark.parametrize("where", ["largest", "smallest"])
def test_close_logits_are_told_apart(where):
    """Two experts whose logits differ in the last bit of one product.  Where that is the largest of x (about 3.5), they differ by 3.5 *
    2^-22: far below the step of an fp32 sum of about 2048 (2^-12), far above a 64-bit one's (2^-41).  Where it is the smallest (about
    2^-11, its last bit 2^-34) they differ by 2^-45, which no 64-bit sum of that size holds: either may come."""
    c, x, a = case([6], 1, E=8, k=1, hidden=2048, inner=256, gate_type=Q4_K, down_type=Q4_K)
    c["router"][:] = 0
    c["router"][2] = c["router"][5] = np.abs(x[0])
    i = int((np.argmax if where == "largest" else np.argmin)(np.abs(x[0])))
    x[0] = np.abs(x[0])
    c["router"][5, i] = np.nextafter(c["router"][5, i], np.float32(np.inf))
    y, ids, p = call(c, dev(x), dev(a))
    if where == "largest":
        assert ids.tolist() == [[5]]
        check(c, x, a, (y, ids, p))
    else:
        assert ids.tolist() in ([[2]], [[5]])


def test_strides_in_place_and_outputs_left_out():
    c, x, a = case([8], 3, E=7, k=3, hidden=512, inner=256, gate_type=Q6_K, down_type=Q4_K)
    layer = device_layer(c)
    y, ids, p = call(c, dev(x), dev(a), layer)
    wide = torch.full((3, 2 * 512 + 8), 5.0, device="cuda")
    wide[:, :512], wide[:, 512:1024] = dev(x), dev(a)
    got, _, _ = call(c, wide[:, :512], wide[:, 512:1024], layer, y=wide[:, 512:1024], ids=False)    # y in add's place
    assert torch.equal(got, y) and torch.equal(wide[:, :512], dev(x)) and (wide[:, 1024:] == 5).all()


def test_not_finite():
    """A token with a NaN or an infinity keeps valid ids, and the others their results; experts that are not chosen may hold anything."""
    c, x, a = case([9], 4, E=12, k=3, hidden=512, inner=512, gate_type=Q4_K, down_type=Q6_K)
    y0, ids0, p0 = call(c, dev(x), dev(a))
    used = set(ids0.flatten().tolist())
    for e in set(range(12)) - used:
        c["gate"][e, :, 0:4] = 0xFF                                        # fp16 NaN scales
        c["down"][e, :, 208:210] = 0xFF
    x2 = x.copy()
    x2[1, 100], x2[2, 7] = np.nan, np.inf
    y, ids, p = call(c, dev(x2), dev(a))
    for t in (0, 3):
        assert torch.equal(y[t], y0[t]) and torch.equal(ids[t], ids0[t]) and torch.equal(p[t], p0[t])
    assert ((ids >= 0) & (ids < 12)).all() and all(len(set(r)) == 3 for r in ids.tolist())
    assert y[1].isnan().all()


def test_extreme_logits():
    """Logits far apart: the others' scores are 0, and a sigmoid's too."""
    for score in (0, 1):
        c, x, a = case([10, score], 1, E=9, k=3, hidden=256, inner=256, gate_type=Q4_K, down_type=Q4_K, score=score, renorm=True)
        c["router"] *= np.float32(2000)
        y, ids, p = call(c, dev(x), dev(a))
        check(c, x, a, (y, ids, p))


def test_graph_replays():
    c, x, a = case([11], 3, E=10, k=4, hidden=512, inner=256, gate_type=Q4_K, down_type=Q6_K)
    layer, xd, ad, y = device_layer(c), dev(x), dev(a), torch.zeros(3, 512, device="cuda")
    n = kq.kqstep_moe_workspace_bytes(layer, 3)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ids, p = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, device="cuda")
    run = lambda: kq.kqstep_moe(layer, 3, xd, 512, ad, 512, y, 512, ids, p, ws, n)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]                    # two graphs over one workspace
    for g in graphs:
        with torch.cuda.graph(g):
            run()
    rng = np.random.default_rng(12)
    for i in range(4):
        xd.copy_(dev(rng.standard_normal((3, 512)).astype(np.float32)))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        check(c, xd.cpu().numpy(), a, (y, ids, p))


def test_streams_side_by_side():
    c, x, a = case([13], 4, E=16, k=4, hidden=1024, inner=512, gate_type=Q4_K, down_type=Q6_K)
    layer = device_layer(c)
    want = call(c, dev(x), dev(a), layer)
    torch.cuda.synchronize()
    n = kq.kqstep_moe_workspace_bytes(layer, 4)
    runs = []
    for _ in range(3):
        s = torch.cuda.Stream()
        runs.append((s, dev(x), dev(a), torch.zeros(4, 1024, device="cuda"), torch.zeros(4, 4, dtype=torch.int32, device="cuda"),
                     torch.zeros(4, 4, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, xd, ad, y, ids, p, ws in runs:
            kq.kqstep_moe(layer, 4, xd, 1024, ad, 1024, y, 1024, ids, p, ws, n, stream=s)
    torch.cuda.synchronize()
    for s, xd, ad, y, ids, p, ws in runs:
        assert torch.equal(y, want[0]) and torch.equal(ids, want[1]) and torch.equal(p, want[2])


def test_refused_tensors():
    c, x, a = case([14], 2, E=4, k=2, hidden=256, inner=256, gate_type=Q4_K, down_type=Q4_K)
    layer = device_layer(c)
    n = kq.kqstep_moe_workspace_bytes(layer, 2)
    y = torch.full((2, 256), 3.0, device="cuda")
    kw = dict(layer=layer, T=2, x=dev(x), ldx=256, add=dev(a), ldadd=256, y=y, ldy=256, ids=torch.zeros(2, 2, dtype=torch.int32, device="cuda"),
              weights=torch.zeros(2, 2, device="cuda"), workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"), workspace_bytes=n)
    for bad in (dict(x=dev(x).cpu()), dict(x=dev(x).half()), dict(add=dev(a).double()), dict(y=y[:, ::2]), dict(ids=kw["ids"].long()),
                dict(weights=kw["weights"].half()), dict(workspace=kw["workspace"].cpu()), dict(add=dev(a).t())):
        with pytest.raises(ValueError):
            kq.kqstep_moe(**dict(kw, **bad))
    assert (y == 3).all()
    for bad in (dict(gate=dev(c["gate"])[:2]), dict(down=torch.zeros(16, dtype=torch.uint8)), dict(router=dev(c["router"]).half()),
                dict(router=dev(c["router"])[:, :64]), dict(bias=torch.zeros(2, device="cuda"))):
        w = dict(E=4, k=2, hidden=256, inner=256, gate_type=Q4_K, gate=dev(c["gate"]), up=dev(c["up"]), down_type=Q4_K, down=dev(c["down"]), router=dev(c["router"]))
        with pytest.raises(ValueError):
            kq.MoELayer(**dict(w, **bad))
