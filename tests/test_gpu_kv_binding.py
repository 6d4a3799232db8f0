"""GPU: the paged-cache binding's checks of real tensors, each refused before
anything is launched, and what the checks let through."""
import numpy as np
import pytest

import kv_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402
from test_gpu_kv import F16, attn_case, check_attn, dev, device_cache, i32, zeros  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_tensors_that_are_not_what_a_call_takes():
    rng = np.random.default_rng(2)
    ref, table, start, q = attn_case(rng, F16, 4, 2, 64, 16, [70, 9], [2, 1])
    cache = device_cache(ref)[0]
    T, n, S = q.shape[0], 4 * 64, table.shape[1]
    out = torch.full((T, n), 3.0, device="cuda")
    ws = torch.empty(max(16, kq.kqkv_attn_workspace_bytes(cache, 2, 2, 70, 4)), dtype=torch.uint8, device="cuda")
    kw = dict(cache=cache, B=2, max_q=2, max_ctx=70, ctx_len=i32([70, 9]), seq_start=i32(start), table=i32(table), table_stride=S, q_heads=4,
              T=T, q=dev(q), ldq=n, scale=0.125, window=0, out=out, ldo=n, workspace=ws, workspace_bytes=ws.numel(), err_flag=zeros(1))
    wide = torch.zeros(2, 2 * S, dtype=torch.int32, device="cuda")
    wide[:, :S] = kw["table"]
    for bad in (dict(table=kw["table"].long()), dict(ctx_len=kw["ctx_len"].long()), dict(table=wide[:, :S]), dict(table=wide[:, ::2]),
                dict(seq_start=kw["seq_start"].cpu()), dict(err_flag=torch.zeros(1, dtype=torch.int32)), dict(err_flag=torch.zeros(1, device="cuda")),
                dict(q=kw["q"].half()), dict(q=kw["q"].double()), dict(out=out.cpu()), dict(out=out.t()), dict(workspace=ws.cpu()),
                dict(workspace=torch.empty(2 * ws.numel(), dtype=torch.uint8, device="cuda")[::2])):
        with pytest.raises(ValueError):
            kq.kqkv_attn(**dict(kw, **bad))
    assert (out == 3).all()
    # rows of wider buffers, at the strides that the call says; another stream
    both = torch.full((T, 2 * n), 3.0, device="cuda")
    both[:, :n] = kw["q"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kq.kqkv_attn(**dict(kw, q=both[:, :n], ldq=2 * n, out=both[:, n:], ldo=2 * n, table=wide[:, :S], table_stride=2 * S), stream=side)
    side.synchronize()
    want, tol = kv_ref.attn(ref, table, [70, 9], start, q, 4, 0.125, 0, out=np.full_like(q, 3.0))
    check_attn(both[:, n:].cpu().numpy(), want, tol)
    slots = i32(np.arange(4))
    for k, v in ((torch.zeros(4, 128, device="cuda", dtype=torch.float16), None), (None, torch.zeros(128, 4, device="cuda").t())):
        with pytest.raises(ValueError):
            kq.kqkv_load(cache, 4, slots, k, v)
    with pytest.raises(ValueError):
        kq.kqkv_load(cache, 4, slots.long(), torch.zeros(4, 128, device="cuda"))
