"""GPU: kqstep_sample against 64 bits: filters and their combinations, ties, masks,
sizes, odd rows, graphs."""
import numpy as np
import pytest

import step_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu
INF = np.float32(np.inf)
LOW = np.finfo(np.float32).min


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a, dtype=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def call(l, t=None, k=None, p=None, mp=None, u=None, pad=0, probs=True, offset=0):
    """l [M][V] (numpy) -> tokens, probabilities.  Rows pad + V apart, `offset` floats into their buffer, NaN and infinities around them."""
    M, V = l.shape
    b = torch.full((offset + M * (V + pad) + 4,), float("inf"), device="cuda")
    rows = b[offset:offset + M * (V + pad)].view(M, V + pad)
    rows[:, V:] = float("nan")
    rows[:, :V] = dev(l)
    u = np.full(M, 0.5, np.float32) if u is None else u
    tokens = torch.full((M + 1,), -9, dtype=torch.int32, device="cuda")
    out = torch.full((M + 1,), 9.0, device="cuda") if probs else None
    n = kq.kqstep_sample_workspace_bytes(M, V)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    kq.kqstep_sample(M, V, rows[:, :V], V + pad, dev(t, np.float32), dev(k, np.int32), dev(p, np.float32), dev(mp, np.float32), dev(u, np.float32),
                     tokens, out, ws, n)
    assert tokens[M] == -9 and (out is None or out[M] == 9)
    return tokens[:M].cpu().numpy(), out[:M].cpu().numpy() if probs else None


def check(l, t=None, k=None, p=None, mp=None, u=None, **kw):
    M = len(l)
    u = np.full(M, 0.5, np.float32) if u is None else np.asarray(u, np.float32)
    tokens, probs = call(l, t, k, p, mp, u, **kw)
    at = lambda a, i, none: none if a is None else a[i]  # noqa: E731
    for i in range(M):
        want, prob, kept = step_ref.sample(l[i], at(t, i, 1.0), at(k, i, 0), at(p, i, 2.0), at(mp, i, 0.0), u[i])
        assert tokens[i] == want, (i, tokens[i], want, kept)
        # rounded once; weights and so their sum are off by at most 2^-36 (half a step of 36 bits of mantissa) and 2^-41 of themselves, or
        # left out 2^-63 below the largest: with both in a quotient, 2 (2^-36 + 2^-41) < 2^-34 of it and 2^-62 a token
        assert probs is None or abs(probs[i] - prob) <= prob * (2.0 ** -24 + 2.0 ** -34) + kept * 2.0 ** -62, (i, probs[i], prob)
    return tokens


def logits(rng, M, V, spread=2.5):
    l = (rng.standard_normal((M, V)) * spread).astype(np.float32)
    for r in l:
        r[rng.integers(0, V, 10)] += rng.uniform(0, 9, 10).astype(np.float32)
    return l


SIZES = [1, 2, 3, 63, 64, 65, 255, 257, 1000, 4095, 4096, 4097, 8193, 32000, 50257, 65537, 128256, 151937, 262144, 300001]


@pytest.mark.parametrize("V", SIZES)
def test_sizes(V):
    rng = np.random.default_rng(V)
    M = 12
    l = logits(rng, M, V)
    check(l, t=[0.8] * M, k=[40] * M, p=[0.95] * M, mp=[0.05] * M, u=rng.random(M))
    check(l, u=rng.random(M))
    check(l, t=[0, 1, 0.1, 0.5, 1.5, 3, 10, 0.7, 1, 1, 1, 1], k=[0, 1, 2, 10, 100, 1000, 5000, V, V - 1, V + 1, -1, 50],
          p=[1, 1, 0.9, 0.5, 0.999, 0.1, 0.7, 0.99, 0.3, 1.5, 0.0, 1], mp=[0, 0, 0.1, 0.0, 0.01, 0.5, 0, 0, 0, 1e-4, 0, 2.0], u=rng.random(M))


def test_largest_vocabulary():
    rng = np.random.default_rng(0)
    l = logits(rng, 3, 1 << 20)
    check(l, t=[1.0, 5.0, 100.0], k=[0, 70000, 0], p=[0.9, 1.0, 0.5], mp=None, u=rng.random(3))


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 2), (64, 3), (5, 1)])
def test_rows_anywhere(pad, offset):
    rng = np.random.default_rng(pad)
    for V in (5, 4097, 33333):
        l = logits(rng, 5, V)
        check(l, t=[0.9] * 5, k=[20, 0, 0, 500, 3], p=[1, 0.8, 1, 0.9, 0.5], mp=[0, 0, 0.02, 0, 0], u=rng.random(5), pad=pad, offset=offset)


def test_one_filter_at_a_time_and_all_draws():
    """The kept set as a whole: draws over a fine grid of u reach each kept token, and none else."""
    rng = np.random.default_rng(4)
    V, M = 300, 2000
    row = logits(rng, 1, V)[0]
    l, u = np.repeat(row[None], M, 0), (np.arange(M) + 0.5) / M
    for kw in (dict(k=[7] * M), dict(p=[0.6] * M), dict(mp=[0.05] * M), dict(k=[30] * M, p=[0.8] * M, mp=[0.01] * M), {}):
        got = set(check(l, t=[1.5] * M, u=u, **kw).tolist())
        n = step_ref.sample(row, 1.5, kw.get("k", [0])[0], kw.get("p", [2.0])[0], kw.get("mp", [0.0])[0], 0.5)[2]
        assert len(got) <= n and (n > 20 or len(got) == n)


@pytest.mark.parametrize("V", [10, 5000, 40000])
def test_ties(V):
    """Equal logits: the lower index first, in every filter."""
    rng = np.random.default_rng(V)
    M = 9
    l = np.zeros((M, V), np.float32)
    l[1] = -0.0
    l[1, ::3] = 0.0
    l[2] = rng.integers(0, 3, V)
    l[3] = np.float32(1e30)
    l[4] = -np.float32(1e30)
    l[5] = rng.integers(0, 2, V) * np.float32(0.001)
    l[6] = rng.integers(-40, 3, V)
    l[7] = 1e-42
    l[7, ::2] = 2e-42
    l[8] = LOW
    k1, k2 = max(1, V // 3), max(1, V // 2 + 1)
    check(l, u=rng.random(M))
    check(l, k=[k1] * M, u=rng.random(M))
    check(l, k=[k2] * M, p=[0.3] * M, u=rng.random(M))
    check(l, p=[0.37] * M, u=rng.random(M), t=[2.0] * M)
    check(l, t=[0.0] * M)
    check(l, k=[1] * M, u=rng.random(M))


def test_masked_rows():
    rng = np.random.default_rng(6)
    V = 9000
    l = logits(rng, 14, V)
    l[0] = -INF
    l[1] = np.nan
    l[2, 1:] = -INF
    l[3, :-1] = np.nan
    l[4, rng.random(V) < 0.99] = -INF
    l[5, rng.random(V) < 0.99] = LOW
    l[6] = LOW
    l[7, 5] = l[7, 4097] = INF
    l[8, ::2] = np.nan
    l[9, 3] = np.float32(3e38)
    l[10] = -INF
    l[10, 100] = LOW
    l[11, :4096] = -INF
    l[12, 4096:] = -INF
    l[13, ::2], l[13, 1::2] = -INF, np.nan
    M = len(l)
    for kw in ({}, dict(k=[50] * M), dict(p=[0.9] * M), dict(mp=[0.1] * M), dict(t=[0.0] * M), dict(t=[1e-30] * M), dict(t=[np.inf] * M),
               dict(t=[np.inf] * M, k=[3000] * M, p=[0.5] * M), dict(k=[V - 1] * M, p=[0.999] * M, mp=[1e-6] * M)):
        got = check(l, u=rng.random(M), **kw)
        assert got[0] == got[1] == got[13] == -1 and got[2] == 0 and got[3] == V - 1 and got[10] == 100


def test_settings_out_of_their_ranges():
    rng = np.random.default_rng(7)
    l = logits(rng, 8, 3000)
    nan = np.nan
    tokens, probs = call(l, t=[nan, -1, 1, 1, 1, 1, 1, 1], k=[0] * 8, p=[1, 1, nan, -1, 0, 1, 1, 1], mp=[0, 0, 0, 0, 0, nan, -1, 5], u=[0.5] * 8)
    first = l.argmax(1)
    for i in (0, 1, 3, 4, 7):                                              # greedy, or nothing but the first token stays
        assert tokens[i] == first[i] and probs[i] == 1
    for i in (2, 5, 6):                                                    # no filter
        assert tokens[i] == step_ref.sample(l[i], 1, 0, 2, 0, 0.5)[0]
    edge, _ = call(np.repeat(l[:1], 5, 0), u=[0.0, -1.0, nan, 1.0, 7.0])
    last = int(np.nonzero(np.exp(l[0].astype(np.float64) - l[0].max()) * 2.0 ** 42 >= 0.5)[0][-1])
    assert list(edge) == [0, 0, 0, last, last]


@pytest.mark.parametrize("V,k,p", [(100, 0, 1.0), (100, 60, 1.0), (100, 0, 1 - 2.0 ** -24), (9000, 0, 1.0), (9000, 5000, 1.0), (9000, 0, 1 - 2.0 ** -24),
                                   (30000, 400, 1.0), (30000, 20000, 1.0)])
def test_u_of_zero_takes_the_first_token_kept(V, k, p):
    """However little it weighs, down to 64 octaves below the largest."""
    rng = np.random.default_rng(V + k)
    octaves = [1, 20, 40, 50, 55, 58, 60, 61, 62]
    M = len(octaves)
    l = np.full((M, V), -np.inf, np.float32)
    for i, o in enumerate(octaves):
        there = rng.permutation(V - 2)[:min(V - 2, 300 if k < 1000 else 15000)] + 2
        l[i, there] = rng.uniform(-2, 0, len(there))
        l[i, V - 1] = 0
        l[i, 1] = -o * np.log(2)
    check(l, t=np.ones(M), k=None if not k else np.full(M, k), p=None if p == 1 else np.full(M, p), u=np.zeros(M))


@pytest.mark.parametrize("V", [40, 3000, 30000])
def test_min_p_far_below_the_largest(V):
    """Borders 20 to 30 octaves down, with logits a few 2^-20 of a weight to each side of them: what is kept shows in the probability of
    the last token at u near 1 (the largest is the first)."""
    M = 8
    l = np.full((M, V), -np.inf, np.float32)
    l[:, 0] = 0
    mp = np.exp(-np.linspace(14, 21, M)).astype(np.float32)
    below = np.log(mp.astype(np.float64))
    for i in range(M):
        # steps of fp32 around the border, at least 2^-19 of it each: none within 2^-24 of it but by chance, which `check` would show
        l[i, 1:] = (below[i] + np.linspace(-3e-5, 3e-5, V - 1)).astype(np.float32)
    for k in (None, np.full(M, min(V - 1, 25)), np.full(M, min(V - 1, 2000))):
        check(l, t=np.ones(M), k=k, mp=mp, u=np.full(M, np.float32(1 - 2.0 ** -24)))


def test_u_at_the_borders_of_tokens():
    """Four tokens of exactly a quarter each: u of a border belongs to the next one."""
    l = np.zeros((8, 4), np.float32)
    u = np.array([0, np.nextafter(np.float32(0.25), np.float32(0)), 0.25, 0.5, np.nextafter(np.float32(0.75), np.float32(0)), 0.75, 0.999, 1 - 2.0 ** -24], np.float32)
    tokens, probs = call(l, u=u)
    assert list(tokens) == [0, 0, 1, 2, 2, 3, 3, 3] and (probs == 0.25).all()


def test_rerun_is_the_same_and_rows_are_by_themselves():
    rng = np.random.default_rng(8)
    l, u = logits(rng, 40, 20000), rng.random(40)
    kw = dict(t=[1.2] * 40, k=[2000] * 40, p=[0.97] * 40)
    a, pa = call(l, u=u, **kw)
    b, pb = call(l, u=u, **kw)
    assert np.array_equal(a, b) and np.array_equal(pa, pb)
    for i in (0, 17, 39):
        c, pc = call(l[i:i + 1], [1.2], [2000], [0.97], None, u[i:i + 1], probs=True)
        assert c[0] == a[i] and pc[0] == pa[i]
    assert np.array_equal(call(l, u=u, probs=False, **kw)[0], a)


def test_no_rows():
    t = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    f = torch.zeros(4, device="cuda")
    kq.kqstep_sample(0, 4, f, 4, None, None, None, None, f, t, None, torch.zeros(16, dtype=torch.uint8, device="cuda"), 16)
    assert t.item() == 5


def test_graph_replays():
    rng = np.random.default_rng(9)
    M, V = 6, 12345
    l, u, tokens, probs = torch.zeros(M, V, device="cuda"), torch.zeros(M, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda"), torch.zeros(M, device="cuda")
    t, k, p = dev([0.7] * M, np.float32), dev([100, 0, 1, 30, 0, 9000], np.int32), dev([0.9, 0.9, 1, 1, 1, 0.5], np.float32)
    n = kq.kqstep_sample_workspace_bytes(M, V)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    run = lambda: kq.kqstep_sample(M, V, l, V, t, k, p, None, u, tokens, probs, ws, n)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            run()
    for i in range(4):
        ln, un = logits(rng, M, V), rng.random(M).astype(np.float32)
        l.copy_(dev(ln)), u.copy_(dev(un))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for j in range(M):
            assert tokens[j].item() == step_ref.sample(ln[j], 0.7, k[j].item(), p[j].item() if p[j].item() < 1 else 2.0, 0.0, un[j])[0]


def test_refused_tensors():
    l, f = torch.zeros(2, 100, device="cuda"), torch.zeros(2, device="cuda")
    i = torch.full((2,), 5, dtype=torch.int32, device="cuda")
    ws = torch.zeros(kq.kqstep_sample_workspace_bytes(2, 100), dtype=torch.uint8, device="cuda")
    kw = dict(M=2, V=100, logits=l, ld=100, temperature=f, top_k=torch.zeros(2, dtype=torch.int32, device="cuda"), top_p=f, min_p=f, u=f, tokens=i, probs=None,
              workspace=ws, workspace_bytes=ws.numel())
    for bad in (dict(logits=l.half()), dict(logits=l.cpu()), dict(logits=l.t()), dict(temperature=f.double()), dict(top_k=f), dict(top_p=f.cpu()), dict(tokens=f),
                dict(u=torch.zeros(4, device="cuda")[::2]), dict(probs=i),
                dict(logits=torch.zeros(2, 208, device="cuda")[:, :100], ld=104)):
        with pytest.raises(ValueError):
            kq.kqstep_sample(**dict(kw, **bad))
    assert (i == 5).all()
