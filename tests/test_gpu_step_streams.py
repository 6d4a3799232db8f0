"""GPU: two whole steps side by side on two streams, round after round, each round from
outputs and workspaces that hold nothing of the one before."""
import pytest

import test_gpu_step_together as together

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def wipe(s):
    for t in [s.y, s.logits, s.probs] + [v for b in s.b for v in b.values() if v.dtype == torch.float32]:
        t.fill_(float("nan"))
    for t in [s.tokens] + [b["ids"] for b in s.b]:
        t.fill_(-5)
    for w in s.ws:
        w.fill_(0x7F)


@pytest.mark.parametrize("sizes", [(2, 5), (8, 1), (8, 8)])
def test_two_steps_on_two_streams(sizes):
    steps = [together.Step(T) for T in sizes]
    want = []
    for s in steps:
        s.run()
        want.append(s.outputs())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for i in range(5):
        for s in steps:
            wipe(s)
        torch.cuda.synchronize()
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(a, b) for a, b in zip(s.outputs(), w)), i
            assert s.err.item() == 0
