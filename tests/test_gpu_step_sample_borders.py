"""GPU: kqstep_sample over rows of many shapes where min_p keeps the tokens that equal
the largest, or those down to a part of it: every row's token and probability are
held against 64 bits, but for the few that a filter's border decides within a rounding."""
import numpy as np
import pytest

import step_ref
import test_gpu_step_shapes as shapes

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def near_a_border(l, t, k, p, mp, u):
    """As in test_gpu_step_shapes, but a token that weighs what the first does is never near min_p's border: up to a min_p of 1 it stays,
    past it only the first does."""
    if shapes.near_a_border(l, t, k, p, 0.0, 1.0):
        return True
    x = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    there = x[x > -np.inf]
    if not t > 0 or not len(there):
        return False
    with np.errstate(all="ignore"):
        w = np.where(there == there.max(), 1.0, np.exp((there - there.max()) / t))
    w[np.isnan(w)] = 0
    e = 2.0 ** -34
    if mp > 0 and (np.abs(w[there < there.max()] / mp - 1) < e).any():
        return True
    # u, among the tokens that are kept
    order = np.lexsort((np.arange(len(x)), -x))
    n = step_ref.sample(l, t, k, p, mp, u)[2]
    kept = np.zeros(len(x))
    with np.errstate(all="ignore"):
        v = np.where(x[order] == x[order[0]], 1.0, np.exp((x[order] - x[order[0]]) / t))
    v[np.isnan(v)] = 0
    kept[order[:n]] = v[:n]
    cum = np.cumsum(kept)
    return bool((np.abs(cum / cum[-1] - u) < e).any())


@pytest.mark.parametrize("V", [5, 300, 8193, 50001, 140000])
@pytest.mark.parametrize("shape", shapes.SHAPES)
def test_rows(shape, V):
    rng = np.random.default_rng([V, shapes.SHAPES.index(shape), 1])
    M = 16
    l = np.stack([shapes.row(shape, V, rng) for _ in range(M)])
    t = rng.choice([0.3, 0.7, 1.0, 1.0, 3.0, 50.0, np.inf], M).astype(np.float32)
    k = rng.choice([0, 0, 0, 40, 600, 5000, 30000], M).astype(np.int32)
    p = rng.choice([1.0, 1.0, 0.5, 0.95], M).astype(np.float32)
    mp = np.resize(np.array([1.0, 1.0, 0.9, np.nextafter(np.float32(1), np.float32(0)), np.nextafter(np.float32(1), np.float32(2)), 0.3, 0.05, np.inf],
                            np.float32), M)
    u = rng.random(M).astype(np.float32)
    d = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    n = kq.kqstep_sample_workspace_bytes(M, V)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    tokens, probs = torch.full((M,), -9, dtype=torch.int32, device="cuda"), torch.full((M,), 9.0, device="cuda")
    kq.kqstep_sample(M, V, d(l), V, d(t), d(k), d(p), d(mp), d(u), tokens, probs, ws, n)
    tokens, probs = tokens.cpu().numpy(), probs.cpu().numpy()
    waived = 0
    for i in range(M):
        want, prob, kept = step_ref.sample(l[i], t[i], k[i], p[i], mp[i], u[i])
        # rounded once; weights of 36 bits of mantissa, in a quotient
        if tokens[i] == want and abs(probs[i] - prob) <= prob * (2.0 ** -24 + 2.0 ** -34) + kept * 2.0 ** -62:
            continue
        args = (float(t[i]), int(k[i]), float(p[i]), float(mp[i]), float(u[i]))
        assert near_a_border(l[i], *args), (i, tokens[i], want, probs[i], prob, args, kept)
        waived += 1
    assert waived <= 2
