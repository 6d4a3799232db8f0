"""GPU: the operators of include/kqstep.h at the ends of their ranges: rows that lie
further apart than 32 bits count, experts past 4 GiB, rows longer than a work-group
keeps, more rows than one launch takes, the largest sizes."""
import numpy as np
import pytest

import step_ref
from kqsynth import Q4_0, Q4_K, Q8_0

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu
FAR = (1 << 31) + 4                               # floats: 8 GiB


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def far_rows(a):
    """a's rows FAR apart; -> the view of them."""
    b = torch.empty((len(a) - 1) * FAR + a.shape[1], device="cuda")
    rows = b.as_strided(a.shape, (FAR, 1))
    rows.copy_(dev(a))
    return rows


def device_layer(c, **kw):
    gate, up, down = (kw[n] if n in kw else dev(c[n]) for n in ("gate", "up", "down"))
    return kq.MoELayer(c["E"], c["k"], c["hidden"], c["inner"], c["gate_type"], gate, up, c["down_type"], down, dev(c["router"]),
                       dev(c["bias"]), c["score"], c["renorm"], c["scale"], c["act"])


def check_moe(c, x, add, layer=None, rows=dev):
    layer = layer or device_layer(c)
    T = len(x)
    n = kq.kqstep_moe_workspace_bytes(layer, T)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    xd, ad, yd = rows(x), rows(add), rows(np.full_like(x, np.nan))
    ids, p = torch.full((T, c["k"]), -7, dtype=torch.int32, device="cuda"), torch.full((T, c["k"]), float("nan"), device="cuda")
    kq.kqstep_moe(layer, T, xd, xd.stride(0), ad, ad.stride(0), yd, yd.stride(0), ids, p, ws, n)
    want, want_ids, want_p, tol = step_ref.moe(c, x, add)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # (computed in 64 bits, rounded once)
    assert (np.abs(p.cpu().numpy() - want_p) <= np.abs(want_p) * (2.0 ** -24 + 2.0 ** -40)).all()
    off = np.abs(yd.cpu().numpy() - want)
    assert (off <= tol).all(), (off / tol).max()


def case(seed, T, **kw):
    rng = np.random.default_rng(seed)
    c = step_ref.layer(rng, **kw)
    return c, rng.standard_normal((T, kw["hidden"])).astype(np.float32), rng.standard_normal((T, kw["hidden"])).astype(np.float32)


@pytest.mark.parametrize("n", [1024, 8192, 65536])
def test_norm_rows_far_apart(n):
    rng = np.random.default_rng(n)
    x, add, w = (rng.standard_normal(s).astype(np.float32) for s in ((2, n), (2, n), n))
    xd, ad = far_rows(x), far_rows(add)
    y = torch.empty(2, n, device="cuda")
    kq.kqstep_norm(2, 1, n, xd, FAR, ad, FAR, ad, FAR, dev(w), 1e-6, y, n)            # (the sum in place)
    h, want = step_ref.norm(x, add, 1, w, 1e-6)
    step_ref.check_norm(y.cpu().numpy(), want)
    assert np.array_equal(ad.cpu().numpy(), h)
    kq.kqstep_norm(2, 1, n, ad, FAR, None, 0, None, 0, dev(w), 1e-6, xd, FAR)
    step_ref.check_norm(xd.cpu().numpy(), want)


def test_norm_most_tokens():
    T = (1 << 23) - 1
    x = torch.randn(T, 4, device="cuda")
    y = torch.empty_like(x)
    kq.kqstep_norm(T, 1, 4, x, 4, None, 0, None, 0, None, 1e-6, y, 4)
    at = np.r_[0:1000, (1 << 21) - 500:(1 << 21) + 500, T - 1000:T]
    step_ref.check_norm(y[at].cpu().numpy(), step_ref.norm(x[at].cpu().numpy(), None, 1, None, 1e-6)[1])
    # the rest against the same in 64 bits on the device: half a step of fp32, and 64-bit roundings
    d = x.double()
    want = d / (d.square().mean(1, keepdim=True) + float(np.float32(1e-6))).sqrt()
    assert ((y.double() - want).abs() <= want.abs() * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -149).all()


def test_moe_rows_far_apart():
    c, x, a = case(1, 2, E=6, k=2, hidden=512, inner=256, gate_type=Q4_K, down_type=Q4_K)
    check_moe(c, x, a, rows=far_rows)


def test_moe_experts_past_4_gib():
    """Only the experts that are chosen are there at all."""
    E, H, F = 1024, 2048, 4096
    c, x, a = case(2, 2, E=3, k=2, hidden=H, inner=F, gate_type=Q8_0, down_type=Q4_0)
    at = [0, 517, E - 1]
    tensors = {}
    for n in ("gate", "up", "down"):
        m = c[n]
        t = torch.empty((E,) + m.shape[1:], dtype=torch.uint8, device="cuda")
        for i, e in enumerate(at):
            t[e] = dev(m[i])
        c[n], tensors[n] = dict(zip(at, m)), t
    assert tensors["gate"].numel() > 1 << 33 and tensors["down"].numel() > 1 << 32
    router = np.zeros((E, H), np.float32)
    router[:] = -np.sign(x[0]) * 0.1              # the others' logits are far below
    router[at] = c["router"]
    c.update(E=E, router=router)
    x[1] = x[0] * np.float32(0.5)
    check_moe(c, x, a, device_layer(c, **tensors))


@pytest.mark.parametrize("H,F,k,T", [(12288, 64, 2, 2), (65536, 32, 1, 1), (64, 1024, 16, 3), (32, 16384, 1, 2), (96, 2048, 5, 8), (12288, 2048, 6, 1)])
def test_moe_rows_longer_than_a_work_group_keeps(H, F, k, T):
    c, x, a = case([H, F], T, E=k, k=k, hidden=H, inner=F, gate_type=Q8_0, down_type=Q8_0)
    check_moe(c, x, a)


@pytest.mark.parametrize("H,F", [(1 << 20, 32), (32, 1 << 20)])
def test_moe_largest_rows(H, F):
    c, x, a = case([H, F, 3], 1, E=1, k=1, hidden=H, inner=F, gate_type=Q4_0, down_type=Q4_0)
    check_moe(c, x, a)


@pytest.mark.parametrize("score", [0, 1])
def test_moe_most_experts(score):
    c, x, a = case([score, 4], 8, E=1024, k=16, hidden=64, inner=32, gate_type=Q4_0, down_type=Q8_0, score=score, renorm=False, bias=True)
    check_moe(c, x, a)
    c, x, a = case([score, 5], 8, E=256, k=16, hidden=64, inner=32, gate_type=Q4_0, down_type=Q8_0, score=score, renorm=False, bias=True)
    c["bias"][200] = np.nan                       # never chosen
    check_moe(c, x, a)


def sampled(l, ld, t, k, p, mp, u):
    M, V = l.shape
    n = kq.kqstep_sample_workspace_bytes(M, V)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    tokens, probs = torch.full((M,), -9, dtype=torch.int32, device="cuda"), torch.full((M,), 9.0, device="cuda")
    kq.kqstep_sample(M, V, l, ld, t, k, p, mp, u, tokens, probs, ws, n)
    return tokens.cpu().numpy(), probs.cpu().numpy()


def check_rows(rows, l, got, t, k, p, mp, u):
    for i in rows:
        want, prob, kept = step_ref.sample(l[i].cpu().numpy(), t[i].item(), k[i].item(), p[i].item(), mp[i].item(), u[i].item())
        assert got[0][i] == want, i
        # rounded once; weights of 36 bits of mantissa, in a quotient
        assert abs(got[1][i] - prob) <= prob * (2.0 ** -24 + 2.0 ** -34) + kept * 2.0 ** -62, i


def settings(M, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pick = lambda v, dtype=torch.float32: torch.tensor(v, dtype=dtype, device="cuda")[torch.randint(0, len(v), (M,), device="cuda", generator=g)]  # noqa: E731
    return (pick([0.0, 0.7, 1.0, 2.0]), pick([0, 3, 40, 400, 900, 3000], torch.int32), pick([0.3, 0.9, 0.99, 1.0]), pick([0.0, 0.0, 0.01, 0.2]),
            torch.rand(M, device="cuda", generator=g))


def test_sample_rows_far_apart():
    rng = np.random.default_rng(3)
    l = far_rows((3 * rng.standard_normal((2, 20001))).astype(np.float32))
    for k in (0, 50):
        s = (torch.full((2,), 0.9, device="cuda"), torch.full((2,), k, dtype=torch.int32, device="cuda"), torch.full((2,), 0.9, device="cuda"),
             torch.zeros(2, device="cuda"), torch.tensor([0.2, 0.9], device="cuda"))
        check_rows(range(2), l, sampled(l, FAR, *s), *s)


@pytest.mark.parametrize("M,V", [(16384, 37), (16385, 200), (40000, 50), (65536, 1), (2048, 70000), (2200, 60000)])
def test_sample_more_rows_than_one_launch_takes(M, V):
    """Each result also by itself: rows of another launch's workspace do not reach it."""
    l = 3 * torch.randn(M, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(M))
    s = settings(M, V)
    got = sampled(l, V, *s)
    rng = np.random.default_rng(M)
    check_rows(np.r_[0, M - 1, rng.integers(0, M, 40 if V > 1000 else 400)], l, got, *s)
    part = slice(M - 300, M)
    again = sampled(l[part], V, *[x[part] for x in s])
    assert np.array_equal(again[0], got[0][part]) and np.array_equal(again[1], got[1][part])


def test_sample_largest_rows():
    M, V = 140, 1 << 20                           # (128 such rows a launch)
    l = 2 * torch.randn(M, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    s = settings(M, 8)
    check_rows([0, 1, 2, 3, 126, 127, 128, 129, 139], l, sampled(l, V, *s), *s)


def test_sample_workspace_does_not_grow_past_a_launch():
    assert kq.kqstep_sample_workspace_bytes(65536, 1 << 20) == kq.kqstep_sample_workspace_bytes(128, 1 << 20) < 400 << 20
    assert kq.kqstep_sample_workspace_bytes(1, 1 << 20) < kq.kqstep_sample_workspace_bytes(2, 1 << 20)
