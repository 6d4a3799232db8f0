"""GPU: kqstep_norm against 64 bits.  Rows of every kernel, strides, in place,
infinities and NaN, Q8_0 rows byte for byte."""
import numpy as np
import pytest

import kv_ref
import step_ref

torch = pytest.importorskip("torch")
import dequant_gemv_gguf_amd as kq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows(rng, T, w, pad):
    """T rows of w inside a buffer whose rows are pad longer, NaN in the padding: the buffer, the rows."""
    b = torch.full((T, w + pad), float("nan"), device="cuda")
    b[:, :w] = dev(rng.standard_normal((T, w)).astype(np.float32) * np.exp(rng.standard_normal((T, 1))).astype(np.float32))
    return b, b[:, :w]


def q8_bytes(y):
    """fp32 rows as their Q8_0 bytes."""
    n, s = kv_ref.quantise(y.reshape(len(y), -1, 32))
    return np.concatenate([s[..., None].view(np.uint8), n.view(np.uint8)], -1).reshape(len(y), -1)


def run(T, heads, n, add, weight, q8, pad, eps=1e-6, seed=0):
    rng = np.random.default_rng([seed, T, heads, n])
    w = heads * n
    xb, x = rows(rng, T, w, pad)
    ab, a = rows(rng, T, w, 2 * pad) if add else (None, None)
    g = rng.standard_normal(n).astype(np.float32) if weight else None
    out = torch.full((2, T + 1, w + pad), 7.0, device="cuda")
    y8 = torch.full((T * w // 32 * 34 + 32,), 77, dtype=torch.uint8, device="cuda") if q8 else None
    x0, a0 = x.clone(), a.clone() if add else None
    kq.kqstep_norm(T, heads, n, x, w + pad, a, w + 2 * pad, out[0, :T, :w] if add else None, w + pad, dev(g) if weight else None, eps,
                   out[1, :T, :w], w + pad, y8)
    h, y = step_ref.norm(x0.cpu().numpy(), a0.cpu().numpy() if add else None, heads, g, eps)
    got = out[1, :T, :w].cpu().numpy()
    step_ref.check_norm(got, y)
    assert (out[1, T] == 7).all() and (out[1, :, w:] == 7).all()
    if add:
        assert np.array_equal(out[0, :T, :w].cpu().numpy(), h)
        assert (out[0, T] == 7).all() and (out[0, :, w:] == 7).all()
    if q8:
        assert np.array_equal(y8[:-32].cpu().numpy().reshape(T, -1), q8_bytes(got)) and (y8[-32:] == 77).all()
    # inputs are left, and what lies beside them was not read
    assert torch.equal(x, x0) and (a is None or torch.equal(a, a0)) and xb[:, w:].isnan().all()


SIZES = [4, 60, 64, 68, 128, 132, 256, 260, 512, 516, 1020, 1024, 1028, 2048, 2052, 4096, 4100, 8192, 8196, 16384, 16388, 32768, 32772]


@pytest.mark.parametrize("n", SIZES)
def test_every_kernel(n):
    for T in (1, 3):
        run(T, 1, n, add=T == 3, weight=True, q8=False, pad=4)


@pytest.mark.parametrize("n", [32, 64, 96, 128, 160, 256, 288, 512, 992, 1024, 1056, 2048, 2080, 4096, 8192, 8224, 16384, 32768, 32800])
def test_eight_bit_rows(n):
    run(2, 1, n, add=True, weight=True, q8=True, pad=0)
    run(3, 1, n, add=False, weight=False, q8=True, pad=8)


@pytest.mark.parametrize("T,heads,n", [(1, 32, 128), (5, 9, 96), (250, 5, 64), (7, 3, 36), (2, 1024, 4), (3, 2, 4096), (17, 71, 32)])
def test_heads(T, heads, n):
    run(T, heads, n, add=False, weight=True, q8=n % 32 == 0, pad=12)
    run(T, heads, n, add=True, weight=True, q8=False, pad=0)


def test_largest_row():
    run(2, 1, 1 << 20, add=True, weight=True, q8=True, pad=4)


def test_many_rows():
    run(70000, 1, 64, add=True, weight=True, q8=True, pad=0)


def test_no_rows():
    y = torch.full((4,), 3.0, device="cuda")
    kq.kqstep_norm(0, 1, 4, y, 4, None, 0, None, 0, None, 0.0, y, 4)
    assert (y == 3).all()


@pytest.mark.parametrize("n", [96, 2048, 8192, 40000])
def test_in_place(n):
    rng = np.random.default_rng(n)
    x, a, g = (rng.standard_normal(s).astype(np.float32) for s in ((3, n), (3, n), n))
    h, y = step_ref.norm(x, a, 1, g, 1e-5)
    for where in ("sum over x, y over add", "y over x", "sum over add"):
        xd, ad, other = dev(x), dev(a), torch.zeros(3, n, device="cuda")
        s, o = {"sum over x, y over add": (xd, ad), "y over x": (None, xd), "sum over add": (ad, other)}[where]
        kq.kqstep_norm(3, 1, n, xd, n, ad, n, s, n, dev(g), 1e-5, o, n)
        step_ref.check_norm(o.cpu().numpy(), y)
        assert s is None or np.array_equal(s.cpu().numpy(), h)


def test_heads_in_place_in_a_wider_row():
    """The query heads of fused q, k, v rows: the rest of the row is left."""
    rng = np.random.default_rng(1)
    b = dev(rng.standard_normal((6, 8 * 64 + 256)).astype(np.float32))
    keep = b.clone()
    _, y = step_ref.norm(b[:, :512].cpu().numpy(), None, 8, None, 1e-6)
    kq.kqstep_norm(6, 8, 64, b, 768, None, 0, None, 0, None, 1e-6, b, 768)
    step_ref.check_norm(b[:, :512].cpu().numpy(), y)
    assert torch.equal(b[:, 512:], keep[:, 512:])


@pytest.mark.parametrize("n", [64, 2048])
def test_special_values(n):
    """Zeros, tiny and huge rows, infinities, NaN: 64 bits hold the squares of all of fp32."""
    x = np.zeros((8, n), np.float32)
    x[1] = 1e-42
    x[2] = 3e38
    x[3, 5] = np.inf
    x[4, 7] = np.nan
    x[5, ::2] = 1e-30
    x[6] = -1e-20
    x[7, 0] = 1.0
    for eps in (0.0, 1e-6, 1e-20):
        y = torch.zeros(8, n, device="cuda")
        y8 = torch.zeros(8 * n // 32 * 34, dtype=torch.uint8, device="cuda")
        kq.kqstep_norm(8, 1, n, dev(x), n, None, 0, None, 0, None, eps, y, n, y8)
        _, want = step_ref.norm(x, None, 1, None, eps)
        got = y.cpu().numpy()
        step_ref.check_norm(got, want)
        if eps:
            assert (got[0] == 0).all()
        a, b = y8.cpu().numpy().reshape(8, -1, 34), q8_bytes(got).reshape(8, -1, 34)
        nan = np.isnan(b[..., :2].copy().view(np.float16)[..., 0])
        assert np.array_equal(nan, np.isnan(a[..., :2].copy().view(np.float16)[..., 0]))
        assert np.array_equal(a[..., 2:], b[..., 2:]) and np.array_equal(a[~nan], b[~nan])


def test_only_eight_bit_rows_and_their_values():
    rng = np.random.default_rng(9)
    x = rng.standard_normal((5, 160)).astype(np.float32)
    y8 = torch.zeros(5 * 5 * 34, dtype=torch.uint8, device="cuda")
    kq.kqstep_norm(5, 1, 160, dev(x), 160, None, 0, None, 0, None, 1e-6, None, 0, y8)
    back = torch.zeros(5, 160, device="cuda")
    kq.kq_dequant(kq.KQ_TYPE_Q8_0, y8, 800, back)
    _, y = step_ref.norm(x, None, 1, None, 1e-6)
    b = y.reshape(5, 5, 32)
    step = np.abs(b).max(-1, keepdims=True) / 127
    # a block's scale is off by half an fp16 step (2^-11), its values by half a step of the scale, and by 127 of the scale's error
    assert np.all(np.abs(back.cpu().numpy().reshape(b.shape) - b) <= step * (0.5 + 127 * 2.0 ** -11) * 1.001)


def test_rows_do_not_depend_on_their_call():
    rng = np.random.default_rng(3)
    x = dev(rng.standard_normal((64, 2048)).astype(np.float32))
    y, one = torch.zeros_like(x), torch.zeros(1, 2048, device="cuda")
    kq.kqstep_norm(64, 1, 2048, x, 2048, None, 0, None, 0, None, 1e-6, y, 2048)
    for i in (0, 31, 63):
        kq.kqstep_norm(1, 1, 2048, x[i:i + 1], 2048, None, 0, None, 0, None, 1e-6, one, 2048)
        assert torch.equal(one[0], y[i])


def test_refused_tensors():
    x, y = torch.zeros(4, 64, device="cuda"), torch.full((4, 64), 3.0, device="cuda")
    kw = dict(T=4, heads=1, n=64, x=x, ldx=64, add=None, ldadd=0, sum=None, ldsum=0, weight=torch.ones(64, device="cuda"), eps=1e-6, y=y, ldy=64)
    for bad in (dict(x=x.cpu()), dict(x=x.half()), dict(x=x.t()), dict(weight=torch.ones(64)), dict(weight=torch.ones(64, device="cuda").half()),
                dict(y=y.double()), dict(y=y[:, ::2]), dict(ldx=68, x=torch.zeros(4, 128, device="cuda")[:, :64])):
        with pytest.raises(ValueError):
            kq.kqstep_norm(**dict(kw, **bad))
    assert (y == 3).all()
