"""GPU: what a row of a verify pass does not see never reaches it: infinities and
NaN in the keys and values of the request's later tokens, of those that have
left the row's window, and in other rows' q.  Rows that do see them are compared
where the 64-bit reference is finite; tolerances are kv_ref.attn's."""
import numpy as np
import pytest

import kv_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402
from test_gpu_kv import F16, Q8, attn_case, run_attn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# q_heads, kv_heads, dim, page, contexts, new tokens, window: one and two row tiles a wave, one to four waves of rows,
# tiles that a window's or the newest tokens' edge cuts, whole and in pieces
CASES = [
    (4, 2, 64, 16, [77, 40], [8, 3], 0),
    (2, 2, 32, 48, [33], [2], 0),
    (16, 2, 128, 64, [70, 31], [8, 8], 0),
    (16, 2, 128, 16, [130, 300], [8, 5], 37),
    (8, 1, 256, 16, [100], [8], 33),
    (6, 1, 160, 32, [45], [4], 9),
    (10, 2, 96, 16, [61], [7], 0),
    (8, 1, 64, 16, [3000], [8], 0),
    (3, 1, 224, 16, [2100], [8], 1000),
    (8, 1, 128, 16, [2500], [8], 600),
]


def edges(ctx, n, window):
    """Tokens of a request that some of its rows see and others do not: the last, one in the middle, the oldest."""
    at = {ctx - 1, ctx - n // 2}
    if window:
        at |= {max(0, ctx - n - window + 1), max(0, ctx - 1 - window)}
    return sorted(at)


def check(ref, table, ctx, start, q, q_heads, scale, window):
    got = run_attn(ref, table, ctx, start, q, q_heads, scale, window, 8)
    with np.errstate(all="ignore"):
        want, tol = kv_ref.attn(ref, table, ctx, start, q, q_heads, float(np.float32(scale)), window, out=np.full_like(q, 3.0))
    fine = np.isfinite(want)
    assert np.isfinite(got[fine]).all()
    assert (np.abs(got - want)[fine] <= tol[fine]).all()
    return got, fine


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("q_heads,kv_heads,dim,page,ctx,new,window", CASES)
def test_values_that_only_some_rows_see(type, q_heads, kv_heads, dim, page, ctx, new, window, bad):
    rng = np.random.default_rng(sum(ctx) + dim)
    ref, table, start, q = attn_case(rng, type, q_heads, kv_heads, dim, page, ctx, new)
    for b, (c, n) in enumerate(zip(ctx, new)):
        for e, i in enumerate(edges(c, n, window)):
            k, v = rng.standard_normal((2, kv_heads, dim))
            v[-1, (5 + 39 * e) % dim] = bad            # (Q8_0: its block of 32)
            ref.put(table[b, i // page] * page + i % page, k, v)
    got, fine = check(ref, table, ctx, start, q, q_heads, dim ** -0.5, window)
    # and rows that see one have no number in its place
    assert not fine.all() and not np.isfinite(got[~fine]).any()
    if not window:
        assert fine[start[:-1]].all()                  # the first row sees none


def test_large_values_that_only_some_rows_see():
    # Q8_0 values past the fp16 range, in the last token
    rng = np.random.default_rng(3)
    ref, table, start, q = attn_case(rng, Q8, 16, 2, 128, 16, [70], [8])
    k, v = rng.standard_normal((2, 2, 128))
    ref.put(table[0, 69 // 16] * 16 + 69 % 16, k, 1e7 * v)
    got = run_attn(ref, table, [70], start, q, 16, 0.1, 0, 8)
    want, tol = kv_ref.attn(ref, table, [70], start, q, 16, float(np.float32(0.1)), 0, out=np.full_like(q, 3.0))
    rows = np.r_[0:7, 8:11]
    assert (np.abs(got - want)[rows] <= tol[rows]).all()


@pytest.mark.parametrize("bad", [np.inf, np.nan])
@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("q_heads,kv_heads,dim,page,ctx,new,window", CASES[:7])
def test_keys_that_only_some_rows_see(type, q_heads, kv_heads, dim, page, ctx, new, window, bad):
    rng = np.random.default_rng(sum(ctx) + dim)
    ref, table, start, q = attn_case(rng, type, q_heads, kv_heads, dim, page, ctx, new)
    q[start[1] - 1, :dim] = bad                        # the first request's last row, one head
    seen = np.zeros(q.shape[0], bool)                  # rows that see a bad key
    for b, (c, n) in enumerate(zip(ctx, new)):
        for i in {c - 1, max(0, c - n - window + 1) if window else c - 1}:
            k, v = rng.standard_normal((2, kv_heads, dim))
            k[:, 5] = bad
            ref.put(table[b, i // page] * page + i % page, k, v)
            for j in range(n):
                p = c - n + j
                seen[start[b] + j] |= i <= p and (not window or i > p - window)
    got = run_attn(ref, table, ctx, start, q, q_heads, dim ** -0.5, window, 8)
    with np.errstate(all="ignore"):
        want, tol = kv_ref.attn(ref, table, ctx, start, q, q_heads, float(np.float32(dim ** -0.5)), window, out=np.full_like(q, 3.0))
    rows = ~seen
    assert rows[:start[-1]].any() and np.isfinite(want[rows]).all()
    assert (np.abs(got - want)[rows] <= tol[rows]).all()
