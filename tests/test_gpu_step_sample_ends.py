"""GPU: kqstep_sample where its settings and logits are at their ends: min_p that no
weight reaches, filters over thousands of tokens, logits far from zero at low
temperatures.  Outputs hold values beforehand that no row may keep."""
import numpy as np
import pytest

import step_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def call(l, t=None, k=None, p=None, mp=None, u=0.5):
    """l [M][V]; settings: one value, or one a row -> tokens, probabilities."""
    M, V = l.shape
    each = lambda v, dtype: None if v is None else torch.from_numpy(np.broadcast_to(np.asarray(v, dtype), M).copy()).cuda()  # noqa: E731
    n = kq.kqstep_sample_workspace_bytes(M, V)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    tokens, probs = torch.full((M,), -9, dtype=torch.int32, device="cuda"), torch.full((M,), 9.0, device="cuda")
    kq.kqstep_sample(M, V, torch.from_numpy(np.ascontiguousarray(l)).cuda(), V, each(t, np.float32), each(k, np.int32), each(p, np.float32),
                     each(mp, np.float32), each(u, np.float32), tokens, probs, ws, n)
    return tokens.cpu().numpy(), probs.cpu().numpy()


def check(l, t=None, k=None, p=None, mp=None, u=0.5):
    M = len(l)
    tokens, probs = call(l, t, k, p, mp, u)
    at = lambda v, i, none: none if v is None else np.broadcast_to(v, M)[i]  # noqa: E731
    for i in range(M):
        want, prob, kept = step_ref.sample(l[i], at(t, i, 1.0), at(k, i, 0), at(p, i, 2.0), at(mp, i, 0.0), at(u, i, 0.5))
        assert tokens[i] == want, (i, tokens[i], want, kept)
        # rounded once (2^-24); weights, and so their sum, within half a step of 36 bits of mantissa (2^-36) and the series' 2^-41 of
        # themselves, or left out 2^-63 below the largest: both in a quotient, below 2^-34 of it and 2^-62 a token
        assert abs(probs[i] - prob) <= prob * (2.0 ** -24 + 2.0 ** -34) + kept * 2.0 ** -62, (i, probs[i], prob)
    return tokens, probs


def nearly_flat(rng, M, V):
    """All weights alike, the first token of the order in the last chunk."""
    l = (0.1 * rng.standard_normal((M, V))).astype(np.float32)
    l[:, V - 1000] = 1
    return l


@pytest.mark.parametrize("p", [0.5, 0.999])
def test_a_row_without_a_weight_of_min_p_gets_its_first_token(p):
    """Wherever u points: into chunks of thousands of tokens, none of which min_p leaves."""
    l = nearly_flat(np.random.default_rng(1), 9, 20000)
    tokens, probs = call(l, p=p, mp=INF, u=np.arange(9) / 9)
    assert (tokens == 19000).all() and (probs > 0).all() and (probs <= 1).all(), (tokens, probs)


@pytest.mark.parametrize("mp", [INF, 5.0, NAN, -1.0])
@pytest.mark.parametrize("V", [300, 6000, 20000])
def test_min_p_out_of_its_range(V, mp):
    """What no weight reaches leaves the first token alone, with a probability of 1; what is no number filters nothing."""
    rng = np.random.default_rng(V)
    M = 8
    flat = nearly_flat(rng, M, max(V, 1100))[:, -V:]
    for l in (flat, np.zeros((M, V), np.float32), np.full((M, V), np.float32(INF)), np.where(flat < 0, flat, np.float32(7))):
        for k, p in ((None, None), (None, 0.3), (None, 0.999), (200, None), (200, 0.9)) + (((3000, 0.9),) if V == 6000 else ()):
            tokens, probs = check(l, k=k, p=p, mp=mp, u=(np.arange(M) + 0.3) / M)
            if mp > 0:
                assert np.array_equal(tokens, l.argmax(1)) and (probs == 1).all()


@pytest.mark.parametrize("V,k,equal", [(60000, 30000, False), (60000, 59999, False), (151937, 50000, False), (40000, 5000, True), (40000, 39000, True)])
def test_both_filters_over_more_tokens_than_are_kept(V, k, equal):
    """top_k, the sum of what it leaves and top_p, each a reduction over the row; the same bits in every run."""
    rng = np.random.default_rng([V, k])
    M = 6
    l = np.zeros((M, V), np.float32) if equal else (2.5 * rng.standard_normal((M, V))).astype(np.float32)
    kw = dict(t=rng.choice([0.8, 1.0, 3.0], M).astype(np.float32), k=k, p=np.array([0.1, 0.5, 0.9, 0.95, 0.99, 0.999], np.float32),
              mp=np.array([0, 0, 0, 0, 1e-4, INF], np.float32), u=rng.random(M).astype(np.float32))
    tokens, probs = check(l, **kw)
    for _ in range(5):
        again = call(l, **kw)
        assert np.array_equal(again[0], tokens) and np.array_equal(again[1], probs)


@pytest.mark.parametrize("top", [16.0, -11.7, 1e5, 3e-8, -2.0 ** 60, 1e30])
def test_probabilities_of_logits_far_from_zero(top):
    """Two tokens a step or a few apart, the lesser one taken, at temperatures that put its probability just above a power of two, where
    half a step of fp32 is the whole 2^-24 of the tolerance: an error of 2^-28 of a weight shows in one row of a hundred."""
    rng = np.random.default_rng(int(abs(np.log2(abs(top)))))
    M = 1000
    top = np.float32(top)
    step = float(abs(np.float64(top) - np.float64(np.nextafter(top, np.float32(-INF)))))
    apart = rng.integers(1, 4, M) * step
    l = np.stack([np.float64(top) - apart, np.full(M, np.float64(top))], 1).astype(np.float32)
    assert np.array_equal(l[:, 1].astype(np.float64) - l[:, 0], apart)
    prob = 2.0 ** -rng.integers(2, 9, M) * (1 + 2.0 ** -11 * rng.random(M))
    t = (apart / np.log(1 / prob - 1)).astype(np.float32)
    tokens, _ = check(l, t=t, u=0.0)
    assert (tokens == 0).all()


def steps_below(rng, M, V, top, steps):
    """Logits up to `steps` fp32 steps below `top`."""
    step = abs(np.spacing(np.float32(top))) / (2 if np.log2(abs(top)) % 1 == 0 and top > 0 else 1)
    return (np.float64(top) - step * rng.integers(0, steps, (M, V))).astype(np.float32), float(step)


@pytest.mark.parametrize("top", [16.0, -11.7, 1e5, 3e-8, -2.0 ** 60, 1e30])
@pytest.mark.parametrize("V,M", [(3, 2000), (40, 300), (3000, 20), (30000, 8)])
def test_weights_do_not_depend_on_where_the_logits_lie(V, M, top):
    """Logits a few fp32 steps from each other, at temperatures of the order of a step: l / t goes up to 2^27, the weights' ratios are
    those of (l - max) / t alone."""
    rng = np.random.default_rng([V, int(abs(np.log2(abs(top))))])
    l, step = steps_below(rng, M, V, top, 12)
    t = (step * rng.uniform(0.3, 3.0, M)).astype(np.float32)
    u = rng.random(M).astype(np.float32)
    check(l, t=t, u=u)
    check(l, t=t, u=u, k=max(1, V // 3), p=0.9)
    check(l, t=t, u=u, mp=0.01)


@pytest.mark.parametrize("V,part", [(7, 0.6), (300, 0.6), (8192, 0.49), (9000, 0.6), (30000, 0.6)])
def test_largest_logits_at_low_temperatures(V, part):
    """Equal ones share the row, whatever their size; all others weigh nothing."""
    M = 8
    rng = np.random.default_rng(V)
    tops = np.array([3.4e38, 3.4e38, -3.4e38, 1e30, -1e30, 1e15, -1e10, 1e-3], np.float32)
    l = np.where(rng.random((M, V)) < part, tops[:, None], np.nextafter(tops, np.float32(-INF))[:, None]).astype(np.float32)
    l[:, 1] = tops
    l[:, 2] = -INF
    t = np.array([1e-30, 1, 1e-30, 1e-10, 1e-20, 1e-3, 1e-3, 1e-14], np.float32)
    for kw in ({}, dict(k=max(1, V // 2)), dict(p=0.5), dict(mp=0.9), dict(mp=1.0), dict(mp=1.01), dict(k=max(1, V // 4), p=0.7, mp=0.1)):
        check(l, t=t, u=(rng.integers(0, 1000, M) + 0.37) / 1000, **kw)
        check(l, t=t, u=0.99937, **kw)


# The largest logit, and a temperature and a min_p at which the next fp32 number below it weighs just that much or a 2^-26 less, and lies
# within a rounding of its 64-bit eighths of an octave from a multiple of them.
BORDERS = [(15.999999046325684, 7.434761783997601e-08, 2.6865993731917115e-06), (15.999950408935547, 1.0194688826459242e-07, 8.656463614897802e-05),
           (15.999944686889648, 7.419148317922009e-08, 2.6150455596507527e-06), (15.999917030334473, 8.416112962095212e-08, 1.1988899132120423e-05),
           (15.999894142150879, 8.461003631055064e-08, 1.2731785318464972e-05), (15.999892234802246, 1.070541557623983e-07, 0.00013525680697057396),
           (15.99988079071045, 7.978613325576589e-08, 6.440637662308291e-06), (15.999874114990234, 7.920611722056492e-08, 5.900860287511023e-06),
           (15.999845504760742, 1.0317498322365282e-07, 9.676058107288554e-05)]


@pytest.mark.parametrize("V", [2, 200, 3000, 6001, 40000])
def test_min_p_of_a_weight_at_the_border_of_an_eighth_of_an_octave(V):
    """One token above, all others of that weight: kept or not as a whole."""
    top, t, mp = (np.array(v, np.float32) for v in zip(*BORDERS))
    l = np.repeat(np.nextafter(top, np.float32(0))[:, None], V, 1)
    l[:, V // 2] = top
    for p in (None, 1 - 2.0 ** -20):
        for u in (0.0, 0.4, 1 - 2.0 ** -24):
            check(l, t=t, mp=mp, p=p, u=u)
    check(l, t=t, mp=mp, k=max(1, V - 1), u=0.4)
    # and a border that top_p reaches inside the same weight
    share = 1 / (1 + (V - 1) * np.exp((l[:, (V // 2 + 1) % V].astype(np.float64) - top) / t))
    check(l, t=t, mp=mp, p=(share + 0.37 * (1 - share)).astype(np.float32), u=0.999)
