"""GPU: the operators of include/kqstep.h as a decode or verify step uses them, between
the products of kqgemv.h and the paged cache of kqkv.h: residual norm, projections,
norms of the heads, rotation and attention, residual norm, mixture-of-experts layer,
and at the end the output matrix and a sampled token for each row.  Every stage is held
against 64 bits on what the stage before it wrote; a captured step against the eager
one."""
import numpy as np
import pytest

import oracle
import step_ref
from kqsynth import Q4_K, Q6_K

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu

HIDDEN, INNER, E, K, HEADS, KV, D, V, PAGE, LAYERS, EPS = 512, 256, 20, 4, 8, 2, 64, 1003, 16, 2, 1e-6


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def matrix(kind, n, k, rng):
    """Random blocks whose rows give products of about one for unit activations."""
    return step_ref.layer(rng, 1, 1, k, n, kind, kind)["gate"][0]


class Step:
    """A model of LAYERS layers that share their workspaces, and its next T tokens."""

    def __init__(self, T):
        rng = np.random.default_rng(T)
        f32 = dict(dtype=torch.float32, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.T, self.w = T, []
        self.gain = lambda n: (1 + 0.1 * rng.standard_normal(n)).astype(np.float32)
        for i in range(LAYERS):
            m = step_ref.layer(rng, E, K, HIDDEN, INNER, Q4_K, Q6_K, score=i, bias=bool(i), scale=1.5 if i else 1.0)
            self.w.append(dict(moe=m, n1=self.gain(HIDDEN), n2=self.gain(HIDDEN), nq=self.gain(D), nk=self.gain(D),
                               q=matrix(Q4_K, HEADS * D, HIDDEN, rng), k=matrix(Q4_K, KV * D, HIDDEN, rng), v=matrix(Q6_K, KV * D, HIDDEN, rng),
                               o=matrix(Q4_K, HIDDEN, HEADS * D, rng)))
        self.last, self.out = self.gain(HIDDEN), matrix(Q6_K, V, HIDDEN, rng)
        self.d = [{n: dev(a) for n, a in w.items() if n != "moe"} for w in self.w]
        self.moe = [kq.MoELayer(E, K, HIDDEN, INNER, Q4_K, dev(w["moe"]["gate"]), dev(w["moe"]["up"]), Q6_K, dev(w["moe"]["down"]),
                                dev(w["moe"]["router"]), dev(w["moe"]["bias"]) if w["moe"]["bias"] is not None else None, w["moe"]["score"],
                                w["moe"]["renorm"], w["moe"]["scale"], w["moe"]["act"]) for w in self.w]
        self.last_d, self.out_d = dev(self.last), dev(self.out)
        new = lambda *s: torch.full(s, float("nan"), **f32)  # noqa: E731
        self.x0 = dev(rng.standard_normal((T, HIDDEN)).astype(np.float32))
        self.b = [dict(y1=new(T, HIDDEN), q=new(T, HEADS * D), k=new(T, KV * D), v=new(T, KV * D), qn=new(T, HEADS * D),
                       kn=new(T, KV * D), qr=new(T, HEADS * D), a=new(T, HEADS * D), o=new(T, HIDDEN), h2=new(T, HIDDEN), y2=new(T, HIDDEN), x=new(T, HIDDEN),
                       ids=torch.full((T, K), -1, **i32), p=new(T, K)) for _ in range(LAYERS)]
        self.y, self.logits = new(T, HIDDEN), new(T, V)
        self.tokens, self.probs = torch.full((T,), -5, **i32), new(T)
        self.u = dev(rng.random(T).astype(np.float32))
        self.temperature, self.top_k = torch.full((T,), 0.8, **f32), torch.full((T,), 40, **i32)
        self.top_p, self.min_p = torch.full((T,), 0.95, **f32), torch.full((T,), 0.02, **f32)
        # one request; its cache, and where its T tokens go
        pages = (T + PAGE - 1) // PAGE + 1
        self.cache = [kq.KVCache(kq.KQKV_F16, KV, D, PAGE, pages, *[torch.zeros(pages * kq.kqkv_page_bytes(kq.KQKV_F16, KV, D, PAGE),
                                                                               dtype=torch.uint8, device="cuda") for _ in range(2)])
                      for _ in range(LAYERS)]
        self.rope = kq.KVRope(kq.KQKV_ROPE_HALVES, D, 10000.0)
        self.table = torch.arange(pages, **i32).view(1, pages)
        self.pos, self.slots = torch.arange(T, **i32), torch.arange(T, **i32)
        self.ctx, self.start, self.err = torch.full((1,), T, **i32), torch.tensor([0, T], **i32), torch.zeros(1, **i32)
        self.sizes = [max(kq.kqkv_attn_workspace_bytes(self.cache[0], 1, T, T, HEADS), 16), kq.kqstep_moe_workspace_bytes(self.moe[0], T),
                      kq.kqstep_sample_workspace_bytes(T, V)]
        self.ws = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in self.sizes]

    def run(self):
        T, x = self.T, self.x0
        for w, b, moe, cache in zip(self.d, self.b, self.moe, self.cache):
            # (the layer before has added the residual itself)
            kq.kqstep_norm(T, 1, HIDDEN, x, HIDDEN, None, 0, None, 0, w["n1"], EPS, b["y1"], HIDDEN)
            kq.kq_qgemv_multi([Q4_K, Q4_K, Q6_K], [w["q"], w["k"], w["v"]], [HEADS * D, KV * D, KV * D], HIDDEN, b["y1"], T, [b["q"], b["k"], b["v"]])
            kq.kqstep_norm(T, HEADS, D, b["q"], HEADS * D, None, 0, None, 0, w["nq"], EPS, b["qn"], HEADS * D)
            kq.kqstep_norm(T, KV, D, b["k"], KV * D, None, 0, None, 0, w["nk"], EPS, b["kn"], KV * D)
            kq.kqkv_rope_store(cache, self.rope, T, self.pos, T, self.slots, HEADS, b["qn"], HEADS * D, b["qr"], HEADS * D, b["kn"], KV * D, b["v"], KV * D)
            kq.kqkv_attn(cache, 1, T, T, self.ctx, self.start, self.table, self.table.shape[1], HEADS, T, b["qr"], HEADS * D, D ** -0.5, 0, b["a"],
                         HEADS * D, self.ws[0], self.sizes[0], self.err)
            kq.kq_qgemv(Q4_K, w["o"], HIDDEN, HEADS * D, b["a"], T, b["o"])
            kq.kqstep_norm(T, 1, HIDDEN, b["o"], HIDDEN, x, HIDDEN, b["h2"], HIDDEN, w["n2"], EPS, b["y2"], HIDDEN)
            kq.kqstep_moe(moe, T, b["y2"], HIDDEN, b["h2"], HIDDEN, b["x"], HIDDEN, b["ids"], b["p"], self.ws[1], self.sizes[1])
            x = b["x"]
        kq.kqstep_norm(T, 1, HIDDEN, x, HIDDEN, None, 0, None, 0, self.last_d, EPS, self.y, HIDDEN)
        kq.kq_qgemv(Q6_K, self.out_d, V, HIDDEN, self.y, T, self.logits)
        kq.kqstep_sample(T, V, self.logits, V, self.temperature, self.top_k, self.top_p, self.min_p, self.u, self.tokens, self.probs, self.ws[2], self.sizes[2])

    def outputs(self):
        return [t.clone() for b in self.b for t in (b["y1"], b["a"], b["h2"], b["x"], b["ids"], b["p"])] + [
            t.clone() for t in (self.y, self.logits, self.tokens, self.probs)]


def norm_is(y, x, add, heads, weight, h=None):
    want_h, want = step_ref.norm(x.cpu().numpy(), None if add is None else add.cpu().numpy(), heads, weight, EPS)
    step_ref.check_norm(y.cpu().numpy(), want)
    assert h is None or np.array_equal(h.cpu().numpy(), want_h)


def product_is(y, kind, W, x):
    want, s = oracle.gemv(kind, W, len(W), x.shape[1], x.cpu().numpy())
    assert (np.abs(y.cpu().numpy() - want) <= 1e-4 * s + 1e-6).all()


@pytest.mark.parametrize("T", [1, 3, 8])
def test_a_step(T):
    s = Step(T)
    s.run()
    torch.cuda.synchronize()
    assert s.err.item() == 0
    x = s.x0
    for w, b in zip(s.w, s.b):
        norm_is(b["y1"], x, None, 1, w["n1"])
        for n, kind in (("q", Q4_K), ("k", Q4_K), ("v", Q6_K)):
            product_is(b[n], kind, w[n], b["y1"])
        norm_is(b["qn"], b["q"], None, HEADS, w["nq"])
        norm_is(b["kn"], b["k"], None, KV, w["nk"])
        product_is(b["o"], Q4_K, w["o"], b["a"])
        norm_is(b["y2"], b["o"], x, 1, w["n2"], b["h2"])
        y, ids, p, tol = step_ref.moe(w["moe"], b["y2"].cpu().numpy(), b["h2"].cpu().numpy())
        assert np.array_equal(b["ids"].cpu().numpy(), ids)
        # (computed in 64 bits, rounded once)
        assert (np.abs(b["p"].cpu().numpy() - p) <= p * (2.0 ** -24 + 2.0 ** -40)).all()
        assert (np.abs(b["x"].cpu().numpy() - y) <= tol).all()
        x = b["x"]
    norm_is(s.y, x, None, 1, s.last)
    product_is(s.logits, Q6_K, s.out, s.y)
    for t, l in enumerate(s.logits.cpu().numpy()):
        token, prob, kept = step_ref.sample(l, 0.8, 40, 0.95, 0.02, s.u[t].item())
        assert s.tokens[t] == token
        # rounded once; weights of 36 bits of mantissa, in a quotient
        assert abs(s.probs[t].item() - prob) <= prob * (2.0 ** -24 + 2.0 ** -34) + kept * 2.0 ** -62


@pytest.mark.parametrize("T", [1, 8])
def test_a_captured_step(T):
    """Replays follow what the arrays hold; eager steps over the same workspaces in between change nothing."""
    s = Step(T)
    s.run()
    first = s.outputs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    rng = np.random.default_rng(99)
    for i in range(4):
        if i == 2:
            s.x0.copy_(dev(rng.standard_normal((T, HIDDEN)).astype(np.float32)))
            s.u.copy_(dev(rng.random(T).astype(np.float32)))
        for t in [s.y, s.logits, s.probs] + [b[n] for b in s.b for n in ("y1", "h2", "x", "p")]:
            t.fill_(float("nan"))
        for w in s.ws:
            w.fill_(0x7F)
        graph.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        s.run()                                   # the same, eagerly
        for a, b in zip(got, s.outputs()):
            assert torch.equal(a, b)
        if i < 2:
            for a, b in zip(got, first):
                assert torch.equal(a, b)
    assert s.err.item() == 0


def test_two_steps_on_two_streams():
    """Each with workspaces of its own."""
    a, b = Step(2), Step(5)
    a.run(), b.run()
    want = a.outputs() + b.outputs()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                s.run()
    torch.cuda.synchronize()
    for x, y in zip(want, a.outputs() + b.outputs()):
        assert torch.equal(x, y)


def test_two_captured_steps_share_workspaces():
    """Replayed in turn on one stream: a workspace keeps nothing between calls."""
    a, b = Step(8), Step(3)
    assert all(x >= y for x, y in zip(a.sizes, b.sizes))
    b.ws, b.sizes = a.ws, a.sizes
    graphs = []
    for s in (a, b):
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    want = []
    for s in (a, b):
        s.run()
        want.append(s.outputs())
    for i in range(6):
        for s in (a, b):
            for t in [s.y, s.logits, s.probs] + [x["x"] for x in s.b]:
                t.fill_(float("nan"))
        for j in ((0, 1) if i % 2 else (1, 0, 1)):
            graphs[j].replay()
        torch.cuda.synchronize()
        for s, w in zip((a, b), want):
            for x, y in zip(s.outputs(), w):
                assert torch.equal(x, y), i
