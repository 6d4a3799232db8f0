"""CPU checks of include/kqkv.h: the library and the binding have every call it
declares, sizes, and every argument error is reported before any HIP call (each
call below fails validation, or has nothing to do)."""
import ctypes
import os
import re

import numpy as np
import pytest

import dequant_gemv_gguf_amd as kq
import kv_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x10000, 0x10002
TYPE, SHAPE, M, NULL, ALIGN, ARG = -1, -2, -3, -4, -5, -6


def status(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except kq.KQError as e:
        return e.status
    return 0


def test_header_library_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kqkv.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(kqkv_[a-z_0-9]+)\s*\(", text)))
    assert names == ["kqkv_attn", "kqkv_attn_workspace_bytes", "kqkv_load", "kqkv_page_bytes", "kqkv_plan",
                     "kqkv_rope_store"]
    L = ctypes.CDLL(kq.lib_path)
    for n in names:
        assert hasattr(L, n) and hasattr(kq, n)


@pytest.mark.parametrize("type,heads,dim,page", [(1, 8, 128, 16), (8, 8, 128, 16), (1, 1, 32, 256), (8, 3, 96, 48),
                                                 (8, 1024, 256, 256)])
def test_page_bytes(type, heads, dim, page):
    want = heads * page * dim * 2 if type == 1 else heads * page * (dim + dim // 32 * 2)
    assert kq.kqkv_page_bytes(type, heads, dim, page) == want


def test_page_bytes_refusals():
    f = kq.kqkv_page_bytes
    assert status(f, 2, 8, 128, 16) == TYPE
    for bad in ((1, 0, 128, 16), (1, 1025, 128, 16), (1, 8, 0, 16), (1, 8, 80, 16), (1, 8, 288, 16), (1, 8, 128, 8),
                (1, 8, 128, 24), (1, 8, 128, 272), (1, 8, 128, 0)):
        assert status(f, *bad) == SHAPE


def cache(type=1, heads=8, dim=128, page=16, pages=10, k=FAKE, v=FAKE):
    return kq.KVCache(type, heads, dim, page, pages, k, v)


BAD_CACHES = [(dict(type=2), TYPE), (dict(heads=0), SHAPE), (dict(dim=100), SHAPE), (dict(page=20), SHAPE),
              (dict(pages=0), SHAPE), (dict(pages=1 << 27), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL),
              (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 8), ALIGN)]


def test_plan_refusals():
    names = ("ctx_len", "new_len", "table", "held", "held_out", "free_pages", "n_free", "n_free_out", "seq_start",
             "ctx_out")
    base = dict(B=4, page_tokens=16, table_stride=8, n_pages=100, T=4, slots=FAKE, pos=FAKE, err_flag=FAKE,
                **{n: FAKE for n in names})
    f = lambda **kw: status(kq.kqkv_plan, **dict(base, **kw))  # noqa: E731
    assert f(B=0) == f(B=-1) == f(B=65537) == f(T=-1) == f(table_stride=0) == f(table_stride=(1 << 24) + 1) == SHAPE
    assert f(page_tokens=0) == f(page_tokens=17) == f(page_tokens=512) == SHAPE
    assert f(n_pages=0) == f(n_pages=1 << 27) == SHAPE
    for n in names:
        assert f(**{n: None}) == NULL
        assert f(**{n: ODD}) == ALIGN
    assert f(slots=None) == f(pos=None) == NULL
    assert f(slots=ODD) == f(pos=ODD) == f(err_flag=ODD) == ALIGN


def test_rope_store_refusals():
    base = dict(cache=cache(), rope=kq.KVRope(0, 128, 1e4), T=4, pos=FAKE, pos_stride=4, slots=FAKE, q_heads=32, q=FAKE,
                ldq=4096, q_out=FAKE, ldq_out=4096, k=FAKE, ldk=1024, v=FAKE, ldv=1024)
    f = lambda **kw: status(kq.kqkv_rope_store, **dict(base, **kw))  # noqa: E731
    assert f(cache=None) == NULL
    for bad, want in BAD_CACHES:
        assert f(cache=cache(**bad)) == want
    assert f(T=-1) == f(T=1 << 27) == f(q_heads=-1) == f(q_heads=1025) == SHAPE
    R = kq.KVRope
    assert f(rope=R(2, 128, 1e4)) == f(rope=R(0, 128, 0.0)) == f(rope=R(0, 128, -1.0)) == ARG
    assert f(rope=R(0, 128, float("inf"))) == f(rope=R(0, 128, float("nan"))) == ARG
    assert f(rope=R(0, 0, 1e4)) == f(rope=R(0, 63, 1e4)) == f(rope=R(0, 130, 1e4)) == SHAPE
    assert f(rope=R(0, 128, 1e4, [])) == f(rope=R(0, 128, 1e4, [16] * 5)) == ARG
    assert f(rope=R(0, 128, 1e4, [32, 31])) == f(rope=R(0, 128, 1e4, [65, -1])) == f(rope=R(0, 128, 1e4, [65])) == ARG
    assert f(rope=R(0, 128, 1e4, [32, 32]), pos_stride=3) == SHAPE
    assert f(rope=None) == ARG                                         # q without a rotation
    assert f(k=None) == f(v=None) == f(pos=None) == f(slots=None) == f(q=None) == f(q_out=None) == NULL
    assert f(pos=ODD) == f(slots=ODD) == f(rope=R(0, 128, 1e4, None, ODD)) == ALIGN
    for n in ("q", "q_out", "k", "v"):
        assert f(**{n: FAKE + 8}) == ALIGN
    for n, ld in (("ldq", 4096), ("ldq_out", 4096), ("ldk", 1024), ("ldv", 1024)):
        assert f(**{n: ld + 2}) == ALIGN and f(**{n: ld - 4}) == SHAPE and f(**{n: 1 << 41}) == SHAPE
    assert f(ldq=8192) == ARG                                          # in place with two strides
    assert f(T=0, q=None, k=None, v=None, pos=None, slots=None) == 0   # nothing to do
    assert f(q_heads=0, k=None, v=None) == 0


def test_load_refusals():
    f = lambda c=None, T=4, slots=FAKE, k=FAKE, v=FAKE: status(kq.kqkv_load, c or cache(), T, slots, k, v)  # noqa: E731
    assert status(kq.kqkv_load, None, 4, FAKE, FAKE, FAKE) == NULL
    for bad, want in BAD_CACHES:
        assert f(cache(**bad)) == want
    assert f(T=-1) == f(T=1 << 27) == SHAPE
    assert f(slots=None) == NULL
    assert f(slots=ODD) == f(k=FAKE + 8) == f(v=FAKE + 4) == ALIGN
    assert f(T=0) == f(k=None, v=None) == 0


def test_attn_refusals():
    need = kq.kqkv_attn_workspace_bytes(cache(), 4, 1, 4096, 32)
    base = dict(cache=cache(), B=4, max_q=1, max_ctx=4096, ctx_len=FAKE, seq_start=FAKE, table=FAKE, table_stride=256,
                q_heads=32, T=4, q=FAKE, ldq=4096, scale=0.1, window=0, out=FAKE, ldo=4096, workspace=FAKE,
                workspace_bytes=need, err_flag=FAKE)
    f = lambda **kw: status(kq.kqkv_attn, **dict(base, **kw))  # noqa: E731
    assert f(cache=None) == NULL
    for bad, want in BAD_CACHES:
        assert f(cache=cache(**bad)) == want
    assert f(B=0) == f(B=4097) == f(max_ctx=0) == f(max_ctx=1 << 31) == SHAPE
    assert f(max_q=0) == f(max_q=9) == M
    assert f(q_heads=0) == f(q_heads=12) == f(q_heads=2048) == SHAPE
    assert f(table_stride=0) == f(table_stride=(1 << 24) + 1) == f(T=-1) == f(T=1 << 27) == SHAPE
    assert f(window=-1) == f(scale=float("inf")) == f(scale=float("nan")) == ARG
    assert f(ctx_len=None) == f(seq_start=None) == f(table=None) == f(q=None) == f(out=None) == NULL
    assert f(ctx_len=ODD) == f(seq_start=ODD) == f(table=ODD) == f(err_flag=ODD) == f(q=ODD) == f(out=ODD) == ALIGN
    assert f(ldq=4098) == f(ldo=4098) == ALIGN
    assert f(ldq=4092) == f(ldo=4092) == SHAPE
    if need:
        assert f(workspace=None) == NULL and f(workspace=FAKE + 8) == ALIGN and f(workspace_bytes=need - 1) == SHAPE
    assert f(T=0) == 0


def test_workspace_bytes_of_invalid_sizes():
    f = kq.kqkv_attn_workspace_bytes
    assert f(None, 4, 1, 4096, 32) == 0
    assert f(cache(type=5), 4, 1, 4096, 32) == f(cache(), 0, 1, 4096, 32) == f(cache(), 4, 9, 4096, 32) == 0
    assert f(cache(), 4, 1, 0, 32) == f(cache(), 4, 1, 4096, 30) == 0


def test_workspace_grows_with_max_ctx():
    # a buffer for the longest context serves every shorter one, and (checked by the call) every window
    for heads, dim, q_heads, max_q in ((8, 128, 64, 1), (8, 128, 64, 8), (1, 32, 1, 1), (8, 256, 8, 3), (2, 160, 16, 8)):
        c = cache(heads=heads, dim=dim)
        for B in (1, 2, 5, 16, 20, 32, 40, 48, 49, 64, 72, 130, 400, 4096):
            need = [kq.kqkv_attn_workspace_bytes(c, B, max_q, n, q_heads)
                    for n in [*range(1, 4000, 31), *range(4000, 20000, 32), 10 ** 5, 10 ** 6, 2 ** 31 - 1]]
            assert need == sorted(need) and need[-1] > 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        kq.KVCache(1, 1, 32, 16, 2, t, t)
    with pytest.raises(ValueError):
        kq.KVRope(0, 32, 1e4, None, torch.ones(16))
    i = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):
        kq.kqkv_plan(1, i, i, 16, i, 1, i, i, i, 1, i, i, 1, i, i, i, i)
    with pytest.raises(ValueError):
        kq.kqkv_attn(cache(), 1, 1, 16, FAKE, FAKE, FAKE, 1, 8, 1, torch.zeros(1, 1024), 1024, 1.0, 0, FAKE, 1024, FAKE, 1 << 30)


def test_reference_quantises_to_the_nearest_multiple():
    # every quant within half a step, and the layout's indexes a bijection
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 32)).astype(np.float32)
    q, s = kv_ref.quantise(x)
    assert np.all(np.abs(q * s[:, None].astype(np.float64) - x) <= 0.5 * s[:, None].astype(np.float64) * (1 + 2.0 ** -9)
                  + 0.5 * 127 * 2.0 ** -11 * s[:, None].astype(np.float64))
    for type, dim, page in ((1, 96, 48), (8, 64, 32)):
        c = kv_ref.Cache(type, 1, dim, page, 1)
        for v in (False, True):
            at = np.concatenate([c._at(t, v) for t in range(page)])
            assert np.array_equal(np.sort(at), np.arange(page * dim))
        at = np.concatenate([c._scale_at(t) for t in range(page)])
        assert np.array_equal(np.sort(at), np.arange(page * dim // 32))
