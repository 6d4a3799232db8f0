"""GPU: how the attention cuts contexts.  The workspace holds, after a call of
cut requests without a window, the pieces' outputs with their m and l, [item][kv
head][row][dim + 4] floats, and last, per request, the items of its first whole
piece and of its last one, and the number of its pieces."""
import numpy as np
import pytest

import kv_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402
from test_gpu_kv import F16, Q8, attn_case, check_attn, dev, device_cache, i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("type", [F16, Q8])
@pytest.mark.parametrize("B", [1, 2, 5])
def test_no_piece_is_empty(type, B):
    # every number of tiles that is cut into pieces of few tiles; of several requests, the others are shorter
    rng = np.random.default_rng(B)
    dim, longest = 32, 90
    ref, table, start, q = attn_case(rng, type, 1, 1, dim, 64, [32 * longest] * B, [1] * B)
    cache = device_cache(ref)
    qd, sd, td, cut = dev(q), i32(start), i32(table), 0
    for tiles in range(17, longest + 1):
        ctx = [32 * max(1, tiles - 7 * b) - (tiles + b) % 3 for b in range(B)]
        nb = kq.kqkv_attn_workspace_bytes(cache[0], B, 1, max(ctx), 1)
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(qd)
        kq.kqkv_attn(cache[0], B, 1, max(ctx), i32(ctx), sd, td, table.shape[1], 1, q.shape[0], qd, dim, 0.2, 0, out, dim, ws, nb)
        ws = ws.cpu().numpy()
        info, part = ws[-16 * B:].view(np.int32).reshape(B, 4), ws[:-16 * B].view(np.float32).reshape(-1, dim + 4)
        for b in range(B):
            whole, last, pieces = info[b, :3]
            if pieces > 1:
                cut += 1
                items = [*range(whole, whole + pieces - 1), last]
                assert (part[items, dim + 1] > 0).all(), (tiles, b, pieces)
        if tiles % 9 == 0:
            check_attn(out.cpu().numpy(), *kv_ref.attn(ref, table, ctx, start, q, 1, float(np.float32(0.2)), 0))
    assert cut > 50
