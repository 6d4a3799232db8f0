"""GPU: what the attention says through err_flag about rows that it leaves."""
import numpy as np
import pytest

import kv_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402,F401
from test_gpu_kv import F16, Q8, attn_case, check_attn, run_attn, zeros  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("ctx,new", [([60, 9], [1, 5]), ([30, 2000], [6, 1]), ([0, 40], [5, 2]), ([12], [300])])
def test_rows_past_max_q_are_said(type, ctx, new):
    rng = np.random.default_rng(len(ctx))
    ref, table, start, q = attn_case(rng, type, 4, 2, 64, 16, ctx, new)
    for max_q in (1, 4, max(new)):
        if max_q > 8:
            continue
        err = zeros(1)
        got = run_attn(ref, table, ctx, start, q, 4, 0.125, 0, max_q, err=err)
        want, tol = kv_ref.attn(ref, table, ctx, start, q, 4, 0.125, 0, max_q=max_q, out=np.full_like(q, 3.0))
        check_attn(got, want, tol)
        assert err.item() == (max(new) > max_q)
        run_attn(ref, table, ctx, start, q, 4, 0.125, 0, max_q)        # without a flag
