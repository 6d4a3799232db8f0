"""CPU checks of include/kqstep.h: the library and the binding have every call it
declares, sizes, and every argument error is reported before any HIP call (each
call below fails validation, or has nothing to do)."""
import ctypes
import os
import re

import dequant_gemv_gguf_amd as kq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x10000, 0x10002
TYPE, SHAPE, M, NULL, ALIGN, ARG = -1, -2, -3, -4, -5, -6
INF, NAN = float("inf"), float("nan")


def status(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except kq.KQError as e:
        return e.status
    return 0


def test_header_library_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kqstep.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(kqstep_[a-z_0-9]+)\s*\(", text)))
    assert names == ["kqstep_moe", "kqstep_moe_workspace_bytes", "kqstep_norm", "kqstep_sample", "kqstep_sample_workspace_bytes"]
    L = ctypes.CDLL(kq.lib_path)
    for n in names:
        assert hasattr(L, n) and hasattr(kq, n)
    for n, v in (("KQSTEP_SOFTMAX", 0), ("KQSTEP_SIGMOID", 1), ("KQSTEP_SILU", 0), ("KQSTEP_GELU", 1)):
        assert getattr(kq, n) == v and re.search(r"%s = %d\b" % (n, v), text)


def test_norm_refusals():
    base = dict(T=4, heads=2, n=64, x=FAKE, ldx=128, add=FAKE, ldadd=128, sum=FAKE * 2, ldsum=128, weight=FAKE, eps=1e-6, y=FAKE * 3,
                ldy=128, y8=FAKE)
    f = lambda **kw: status(kq.kqstep_norm, **dict(base, **kw))  # noqa: E731
    assert f(T=-1) == f(T=1 << 23) == f(heads=0) == f(heads=1025) == f(n=0) == f(n=-4) == f(n=6) == f(n=1 << 21) == SHAPE
    assert f(heads=1024, n=1028) == SHAPE                              # a row beyond 2^20
    assert f(T=1 << 22, heads=1024, n=4, ldx=4096, ldadd=4096, ldsum=4096, ldy=4096, y8=None) == SHAPE
    assert f(n=36, heads=1) == SHAPE                                   # no whole blocks
    assert f(eps=-1e-6) == f(eps=INF) == f(eps=NAN) == f(add=None) == ARG
    assert f(y=None, y8=None) == f(x=None) == NULL
    for n, ld in (("x", "ldx"), ("add", "ldadd"), ("sum", "ldsum"), ("y", "ldy")):
        assert f(**{n: FAKE * 5 + 8}) == f(**{ld: 130}) == ALIGN
        assert f(**{ld: 124}) == f(**{ld: 1 << 41}) == SHAPE
    assert f(weight=FAKE + 4) == f(y8=FAKE + 2) == ALIGN
    assert f(x=FAKE * 2, ldx=256) == f(sum=FAKE, ldsum=256) == f(y=FAKE, ldy=256) == f(x=FAKE * 3, ldx=256) == ARG   # in place, two strides
    assert f(y=FAKE * 2) == ARG                                        # sum and y in one place
    assert f(T=0, x=None, y=None, y8=None) == 0


def layer(**kw):
    a = dict(E=16, k=4, hidden=512, inner=256, gate_type=12, gate=FAKE, up=FAKE, down_type=14, down=FAKE, router=FAKE, bias=FAKE)
    return kq.MoELayer(**dict(a, **kw))


BAD_LAYERS = [(dict(E=0), ARG), (dict(E=1025), ARG), (dict(k=0), ARG), (dict(k=17, E=32), ARG), (dict(k=5, E=4), ARG),
              (dict(gate_type=3), TYPE), (dict(down_type=1), TYPE), (dict(hidden=0), SHAPE), (dict(hidden=288), SHAPE),
              (dict(hidden=(1 << 20) + 256), SHAPE), (dict(inner=0), SHAPE), (dict(inner=-256), SHAPE), (dict(inner=272), SHAPE),
              (dict(inner=(1 << 20) + 256), SHAPE)]


def test_moe_refusals():
    need = kq.kqstep_moe_workspace_bytes(layer(), 3)
    assert need >= 3 * (16 * 8 + 4 * 256 * 4)
    base = dict(layer=layer(), T=3, x=FAKE, ldx=512, add=FAKE, ldadd=512, y=FAKE * 2, ldy=512, ids=FAKE, weights=FAKE, workspace=FAKE,
                workspace_bytes=need)
    f = lambda **kw: status(kq.kqstep_moe, **dict(base, **kw))  # noqa: E731
    assert f(layer=None) == NULL and kq.kqstep_moe_workspace_bytes(None, 1) == 0
    for bad, want in BAD_LAYERS:
        assert f(layer=layer(**bad)) == want, bad
        assert kq.kqstep_moe_workspace_bytes(layer(**bad), 1) == 0
    assert f(layer=layer(score=2)) == f(layer=layer(act=2)) == f(layer=layer(act=-1)) == f(layer=layer(scale=INF)) == ARG
    assert f(T=0) == f(T=9) == M and kq.kqstep_moe_workspace_bytes(layer(), 0) == kq.kqstep_moe_workspace_bytes(layer(), 9) == 0
    for n in ("gate", "up", "down", "router"):
        assert f(layer=layer(**{n: None})) == NULL and f(layer=layer(**{n: FAKE + 8})) == ALIGN
    assert f(layer=layer(bias=ODD)) == f(ids=ODD) == f(weights=ODD) == f(workspace=FAKE + 8) == ALIGN
    assert f(x=None) == f(y=None) == f(workspace=None) == NULL
    for n, ld in (("x", "ldx"), ("add", "ldadd"), ("y", "ldy")):
        assert f(**{n: FAKE * 5 + 8}) == f(**{ld: 514}) == ALIGN
        assert f(**{ld: 508}) == f(**{ld: 1 << 41}) == SHAPE
    assert f(y=FAKE) == f(add=FAKE * 2, ldadd=1024) == ARG             # y over x; y in add's place with two strides
    assert f(workspace_bytes=need - 1) == SHAPE


def test_sample_refusals():
    need = kq.kqstep_sample_workspace_bytes(4, 1000)
    base = dict(M=4, V=1000, logits=FAKE, ld=1000, temperature=FAKE, top_k=FAKE, top_p=FAKE, min_p=FAKE, u=FAKE, tokens=FAKE, probs=FAKE,
                workspace=FAKE, workspace_bytes=need)
    f = lambda **kw: status(kq.kqstep_sample, **dict(base, **kw))  # noqa: E731
    for m, v in ((-1, 1000), (65537, 1000), (4, 0), (4, (1 << 20) + 1)):
        assert f(M=m, V=v) == SHAPE and kq.kqstep_sample_workspace_bytes(m, v) == 0
    assert f(ld=999) == f(ld=1 << 41) == f(workspace_bytes=need - 1) == SHAPE
    for n in ("logits", "u", "tokens", "workspace"):
        assert f(**{n: None}) == NULL
    for n in ("logits", "temperature", "top_k", "top_p", "min_p", "u", "tokens", "probs"):
        assert f(**{n: ODD}) == ALIGN
    assert f(workspace=FAKE + 8) == ALIGN
    assert f(M=0, logits=None) == 0
