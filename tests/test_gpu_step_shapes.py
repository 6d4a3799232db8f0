"""GPU: kqstep_sample over rows of many shapes, so that every way to a token is taken:
few tokens, lists of the chunks, ordered chunks, the row gone over again, digits over
the whole row."""
import numpy as np
import pytest

import step_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu
SHAPES = ["normal", "descending", "ascending", "quarters", "two values", "uniform", "tail", "one above", "masked", "first chunk", "steps of an octave",
          "far below", "wide", "nearly flat", "equal but for one", "infinities"]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def row(shape, V, rng):
    l = rng.standard_normal(V) * 2.5
    if shape in ("descending", "ascending"):
        l = np.sort(l)[::-1 if shape == "descending" else 1]
    elif shape == "quarters":
        l = np.rint(4 * l) / 4
    elif shape == "two values":
        l = np.where(rng.random(V) < 0.3, 1.5, -0.75)
    elif shape == "uniform":
        l = rng.uniform(-20, 0, V)
    elif shape == "tail":
        l = rng.standard_t(2, V)
    elif shape == "one above":
        l[rng.integers(0, V)] = 30
    elif shape == "masked":
        l[rng.random(V) < 0.99] = [-np.inf, np.nan, np.finfo(np.float32).min][rng.integers(0, 3)]
    elif shape == "first chunk":
        l[:8192] += 12
    elif shape == "steps of an octave":
        l = -np.log(2) * rng.integers(0, 70, V)
    elif shape == "far below":
        l = np.where(rng.random(V) < 0.01, l, l - 60)
    elif shape == "wide":
        l *= 1e6
    elif shape == "nearly flat":
        l *= 1e-6
    elif shape == "equal but for one":
        l = np.full(V, -3.25)
        l[rng.integers(0, V)] += rng.choice([-1, 1]) * 1e-3
    elif shape == "infinities":
        l[rng.random(V) < 0.001] = np.inf
        l[rng.random(V) < 0.2] = -np.inf
    return l.astype(np.float32)


def near_a_border(l, t, k, p, mp, u):
    """Whether a filter or u falls so near to the border of a token that weights of 36 bits decide it: borders move by the weights' and
    sums' errors, 2^-35 of the sum."""
    x = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    if not t > 0 or not (x > -np.inf).any():
        return False
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    with np.errstate(all="ignore"):
        w = np.where(x[order] == x[order[0]], 1.0, np.exp((x[order] - x[order[0]]) / t))
    w[np.isnan(w)] = 0
    e = 2.0 ** -34
    if k > 0:
        w = w[:k]
    if p < 1:
        cum = np.cumsum(w)
        if (np.abs(cum / cum[-1] - p) < e).any():
            return True
    if mp > 0 and (np.abs(w / mp - 1) < e).any():
        return True
    n = step_ref.sample(l, t, k, p, mp, u)[2]
    kept = np.zeros(len(x))
    kept[order[:n]] = w[:n]
    cum = np.cumsum(kept)
    return bool((np.abs(cum / cum[-1] - u) < e).any()) and u < 1


@pytest.mark.parametrize("V", [5, 300, 8191, 8192, 8193, 16385, 50001, 140000])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows(shape, V):
    rng = np.random.default_rng([V, SHAPES.index(shape)])
    M = 24
    l = np.stack([row(shape, V, rng) for _ in range(M)])
    t = rng.choice([0.3, 0.7, 1.0, 1.0, 3.0, 50.0, np.inf], M).astype(np.float32)
    k = rng.choice([0, 0, 0, 1, 2, 40, 256, 400, 512, 600, 1000, 5000, 30000], M).astype(np.int32)
    p = rng.choice([1.0, 1.0, 0.05, 0.5, 0.9, 0.95, 0.999], M).astype(np.float32)
    mp = rng.choice([0.0, 0.0, 0.0, 1e-6, 0.001, 0.05, 0.3, 1.0], M).astype(np.float32)
    u = rng.random(M).astype(np.float32)
    d = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    n = kq.kqstep_sample_workspace_bytes(M, V)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    tokens, probs = torch.full((M,), -9, dtype=torch.int32, device="cuda"), torch.full((M,), 9.0, device="cuda")
    kq.kqstep_sample(M, V, d(l), V, d(t), d(k), d(p), d(mp), d(u), tokens, probs, ws, n)
    tokens, probs = tokens.cpu().numpy(), probs.cpu().numpy()
    decided = 0
    for i in range(M):
        want, prob, kept = step_ref.sample(l[i], t[i], k[i], p[i], mp[i], u[i])
        args = (l[i], float(t[i]), int(k[i]), float(p[i]), float(mp[i]), float(u[i]))
        if tokens[i] != want:
            # borders of equal weights are not exactly where the sums of them are (a third of them is no binary number)
            assert near_a_border(*args), (i, tokens[i], want, args[1:], kept)
            continue
        decided += 1
        # rounded once; weights of 36 bits of mantissa, in a quotient; and a token more or less at a border
        tol = prob * (2.0 ** -24 + 2.0 ** -34) + kept * 2.0 ** -62
        assert abs(probs[i] - prob) <= tol or near_a_border(*args), (i, probs[i], prob, args[1:], kept)
    assert decided >= M - 4
