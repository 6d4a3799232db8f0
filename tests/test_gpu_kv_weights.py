"""GPU: how finely the attention holds a softmax weight that is far below its
row's largest (include/kqkv.h: within 2^-31 of the largest)."""
import numpy as np
import pytest

import kv_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402,F401
from test_gpu_kv import F16, Q8, attn_case, run_attn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("steps", [0.6, 1.9, 3.1, 37.9, 1000.9, 16384.9])
@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("q_heads,dim", [(1, 64), (40, 128), (40, 256)])
def test_a_long_tail_of_small_weights(type, q_heads, dim, steps):
    """Four keys (one in each of the first tiles, so that every wave has one) have the value 0, all others the score 0, the
    value 1 and `steps` 2^-30 of the four's weight w0.  out = N w / (4 w0 + N w): a weight off by 2^-31 w0 puts it off by
    N 2^-31 / (4 + N w / w0).  Beside that, a weight's relative error is that of its exponent and of exp2: the scores of up
    to 31 (in units of ln 2) are off by their scale's two roundings, 31 * 2^-23 at most (q and k are powers of two and
    enter exactly; a Q8_0 scale times a sum that is exact is one more rounding, 2^-24), their difference from the
    running maximum by 2^-19, exp2 by 2^-22, and the sums of 512 terms, four waves, by 20 roundings: 2^-17 in all."""
    n, heads4 = 512 if q_heads == 1 else 256, (0, 32, 64, 96)         # (short enough that none is cut)
    rng = np.random.default_rng(1)
    ref, table, start, q = attn_case(rng, type, q_heads, 1, dim, 16, [n], [1])
    for i in range(n):
        top = i in heads4
        ref.put(table[0, i // 16] * 16 + i % 16, np.full((1, dim), 1.0 if top else 0.0), np.full((1, dim), 0.0 if top else 1.0))
    q[:] = 0.5
    k, v = ref.get(table[0, 0] * 16)[0][0], ref.get(table[0, 0] * 16 + 1)[1][0]
    scale = float(np.float32(-np.log(steps * 2.0 ** -30) / (0.5 * k.sum())))
    w = np.exp(-scale * 0.5 * k.sum())
    assert abs(w * 2.0 ** 30 / steps - 1) < 2.0 ** -19
    want = (n - 4) * w * v / (4 + (n - 4) * w)
    tol = (n - 4) * (2.0 ** -31 + 2.0 ** -17 * w) * v / (4 + (n - 4) * w)
    got = run_attn(ref, table, [n], start, q, q_heads, scale, 0, 1)[0].reshape(q_heads, dim)
    worst = (np.abs(got - want) / tol).max()
    print("steps %g: worst %.3g of the bound" % (steps, worst))
    assert worst <= 1
