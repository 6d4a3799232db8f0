"""GPU: kqstep_moe's choice among experts whose logits differ by the last bits of 64-bit
values, whatever the number of experts."""
import numpy as np
import pytest

import step_ref
from kqsynth import Q4_0, Q8_0

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def chosen(c, x):
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    layer = kq.MoELayer(c["E"], c["k"], c["hidden"], c["inner"], c["gate_type"], dev(c["gate"]), dev(c["up"]), c["down_type"], dev(c["down"]),
                        dev(c["router"]), dev(c["bias"]), c["score"], c["renorm"], c["scale"], c["act"])
    T, H = x.shape
    n = kq.kqstep_moe_workspace_bytes(layer, T)
    ids = torch.full((T, c["k"]), -7, dtype=torch.int32, device="cuda")
    kq.kqstep_moe(layer, T, dev(x), H, None, 0, torch.empty(T, H, device="cuda"), H, ids, None, torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n)
    return ids.cpu().numpy()


COUNTS = [(8, 3), (64, 1), (70, 8), (128, 2), (130, 5), (256, 16), (256, 1), (257, 5), (1000, 4)]


@pytest.mark.parametrize("E,k", COUNTS)
@pytest.mark.parametrize("bits", [46, 49, 52])
def test_logits_that_differ_by_their_last_bits(E, k, bits):
    """Products and sums that 64 bits hold exactly: 1 and 1 + 2^-bits.  Those a bit above come first, the others by their number."""
    c = step_ref.layer(np.random.default_rng([E, k]), E=E, k=k, hidden=64, inner=32, gate_type=Q8_0, down_type=Q4_0)
    x = np.zeros((2, 64), np.float32)
    x[:, 0], x[:, 1] = 1, 2.0 ** -26
    x[1] = -x[1]
    c["router"][:] = 0
    c["router"][:, 0] = 1
    above = [E - 1, E // 2, 5]
    c["router"][above, 1] = 2.0 ** (26 - bits)
    ids = chosen(c, x)
    rest = [e for e in range(E) if e not in above]
    assert ids[0].tolist() == (sorted(above) + rest)[:k] and ids[1].tolist() == (rest + sorted(above))[:k]


@pytest.mark.parametrize("E,k", COUNTS)
def test_scores_with_a_bias_that_differ_by_their_last_bits(E, k):
    c = step_ref.layer(np.random.default_rng([E, k, 1]), E=E, k=k, hidden=64, inner=32, gate_type=Q8_0, down_type=Q4_0, score=1, bias=True)
    c["router"][:] = 0                                                     # a sigmoid of 0: a half
    c["bias"][:] = 0
    c["bias"][E - 2], c["bias"][6] = 2.0 ** -53, 2.0 ** -50
    first = [6, E - 2] if E > 8 else [6]                                   # (E = 8: E - 2 is 6)
    assert chosen(c, np.ones((1, 64), np.float32))[0].tolist() == (first + [e for e in range(E) if e not in first])[:k]


@pytest.mark.parametrize("E,k", COUNTS)
def test_equal_logits_zeros_of_both_signs_and_no_numbers(E, k):
    """Equal ones by their number, NaN after all of them and by number too."""
    c = step_ref.layer(np.random.default_rng([E, k, 2]), E=E, k=k, hidden=64, inner=32, gate_type=Q8_0, down_type=Q4_0)
    c["router"][:] = 0
    c["router"][::2, 3] = -1                                               # -1 * 0: a zero of the other sign
    c["router"][E - 1, 5] = np.nan
    c["router"][0, 5] = np.nan
    x = np.ones((3, 64), np.float32)
    x[:, 3] = 0
    x[2, 7] = np.nan                                                       # every logit
    ids = chosen(c, x)
    assert ids[0].tolist() == ids[1].tolist() == (list(range(1, E - 1)) + [0, E - 1])[:k] and ids[2].tolist() == list(range(k))
