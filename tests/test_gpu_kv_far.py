"""GPU: attention at large scores, with bounds that are far below the outputs,
and the kernels that read long contexts past the caches, at every head size."""
import numpy as np
import pytest

import kv_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402,F401
from test_gpu_kv import F16, Q8, attn_case, check_attn, run_attn  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def keys_of(ref, table, b, n):
    both = [ref.get(table[b, i // ref.page] * ref.page + i % ref.page) for i in range(n)]
    return np.stack([k for k, _ in both]), np.stack([v for _, v in both])


@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("dim,ctx", [(64, 300), (96, 3000), (256, 300)])
def test_one_key_wins(type, dim, ctx):
    """Each query head has a key along its q.  Where that key's score is more than 60 above every other's (asserted), the
    others' weights are e^-60 at most, and the output is that key's value: its weight in two limbs (2^-21), the product's
    and the sums' few roundings, and the division: 2^-20 of each element, and of the others' ctx e^-60 times the largest."""
    rng = np.random.default_rng(dim)
    heads, scale = 4, 1 / np.sqrt(dim)
    ref, table, start, q = attn_case(rng, type, heads, 1, dim, 16, [ctx], [1])
    at = [0, ctx // 2, ctx - 1, 37]
    for h, i in enumerate(at):
        ref.put(table[0, i // 16] * 16 + i % 16, 20 * q[0].reshape(heads, dim)[h:h + 1], rng.standard_normal((1, dim)))
    k, v = keys_of(ref, table, 0, ctx)
    for factor in (1.0, 30.0, 1e4, 1e8):
        x = (q * np.float32(factor)).astype(np.float32)
        got = run_attn(ref, table, [ctx], start, x, heads, scale, 0, 1)[0].reshape(heads, dim)
        for h, i in enumerate(at):
            s = scale * (k[:, 0] @ x[0].reshape(heads, dim)[h].astype(np.float64))
            assert s[i] - np.delete(s, i).max() > 60
            tol = 2.0 ** -20 * np.abs(v[i, 0]) + ctx * np.exp(-60.0) * np.abs(v).max()
            assert (np.abs(got[h] - v[i, 0]) <= tol).all(), (factor, h)


@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("factor", [1.0, 8.0, 64.0])
@pytest.mark.parametrize("dim,ctx", [(64, 400), (160, 1500)])
def test_keys_of_like_scores(type, factor, dim, ctx):
    """Each key's score error is bounded by its own q and k: S_i = scale * sum |q_d k_id| times the limbs' 2^-22, two
    roundings of the scale and dim of the sums (2^-21 + dim u), and three roundings of the exponent at the row's largest
    score, in units of ln 2; its weight's, by that, 2^-21 for exp2 and the limbs, and 2^-31 of the largest weight.  The
    output is off by the weighted mean of those, in the sum of the values and in the sum of the weights, and by the sums'
    (n / 32 + 64) u each."""
    rng = np.random.default_rng(dim)
    heads, scale = 4, 1 / np.sqrt(dim)
    ref, table, start, q = attn_case(rng, type, heads, 1, dim, 16, [ctx], [1])
    x = (q * np.float32(factor)).astype(np.float32)
    got = run_attn(ref, table, [ctx], start, x, heads, scale, 0, 1)[0].reshape(heads, dim)
    k, v = keys_of(ref, table, 0, ctx)
    k, v = k[:, 0], v[:, 0]
    for h in range(heads):
        y = x[0].reshape(heads, dim)[h].astype(np.float64)
        s = scale * (k @ y)
        w = np.exp(s - s.max())
        e = scale * (np.abs(k) @ np.abs(y)) * (2.0 ** -21 + dim * U) + 3 * U * np.abs(s).max() / np.log(2) + 2.0 ** -21
        assert e.max() < 0.05
        e = w * e * 1.05 + 2.0 ** -31
        mean = w @ np.abs(v) / w.sum()
        tol = (e @ np.abs(v) + e.sum() * mean) / w.sum() + 2 * (ctx / 32 + 64) * U * mean
        assert tol.max() < 2e-2 * mean.max()
        assert (np.abs(got[h] - w @ v / w.sum()) <= tol).all(), h


@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("dim", range(32, 257, 32))
def test_hint_of_a_huge_context_at_every_head_size(type, dim):
    rng = np.random.default_rng(dim)
    ctx, new = [1300, 0, 31, 700], [1, 1, 0, 2]
    ref, table, start, q = attn_case(rng, type, 6, 2, dim, 48, ctx, new)
    for window in (0, 500):
        got = run_attn(ref, table, ctx, start, q, 6, dim ** -0.5, window, 2, max_ctx=2 ** 31 - 1)
        want, tol = kv_ref.attn(ref, table, ctx, start, q, 6, float(np.float32(dim ** -0.5)), window, out=np.full_like(q, 3.0))
        check_attn(got, want, tol)
