"""CPU checks of the paged-cache binding with stand-ins for device tensors:
what it keeps alive, and what it refuses before the library is called."""
import gc
import weakref

import pytest

import dequant_gemv_gguf_amd as kq
from dequant_gemv_gguf_amd import _binding as binding

torch = pytest.importorskip("torch")


class Device:
    """What the binding asks a device tensor for, over a host tensor's shape and
    strides and an address that nothing may follow."""

    def __init__(self, t, device=0, at=0x10000):
        self.t, self.device, self.at = t, device, at
        self.is_cuda, self.dtype, self.shape = device is not None, t.dtype, t.shape

    def __getattr__(self, name):
        if name in ("is_contiguous", "numel", "element_size", "stride", "dim", "size"):
            return getattr(self.t, name)
        raise AttributeError(name)

    def get_device(self):
        return -1 if self.device is None else self.device

    def data_ptr(self):
        return self.at


@pytest.fixture(autouse=True)
def devices(monkeypatch):
    """The current device and each device's current stream, without a GPU; what
    of it was asked for and made current."""
    class C:
        current, asked = 0, []

        def _cuda_getDevice():
            return C.current

        def _cuda_getCurrentRawStream(device):
            C.asked.append((C.current, device))
            return 0x7000 + device

    class On:
        def __init__(self, device):
            self.to = device

        def __enter__(self):
            self.before, C.current = C.current, self.to

        def __exit__(self, *_):
            C.current = self.before

    binding._load_torch()
    monkeypatch.setattr(binding, "_torch_c", C)
    monkeypatch.setattr(torch.cuda, "device", On)
    C.asked = []
    return C


def bytes_(n):
    return Device(torch.zeros(n, dtype=torch.uint8))


def collected(make):
    """Whether what `make` returns, and the tensors it was made of, go away with
    the last reference to it."""
    tensors, made = make()
    refs = [weakref.ref(t) for t in tensors]
    del tensors
    assert all(r() is not None for r in refs)       # kept alive by `made`
    del made
    gc.collect()
    return all(r() is None for r in refs)


def test_a_dropped_cache_lets_its_buffers_go():
    def make():
        t = [bytes_(3 * kq.kqkv_page_bytes(kq.KQKV_F16, 2, 64, 16)) for _ in range(2)]
        return t, kq.KVCache(kq.KQKV_F16, 2, 64, 16, 3, *t)
    assert collected(make)


def test_a_dropped_rope_lets_its_factors_go():
    def make():
        t = Device(torch.ones(32))
        return [t], kq.KVRope(kq.KQKV_ROPE_PAIRS, 64, 1e4, None, t)
    assert collected(make)


def test_a_dropped_cache_lets_its_buffers_go_after_calls():
    def make():
        t = [bytes_(3 * kq.kqkv_page_bytes(kq.KQKV_Q8_0, 2, 64, 16)) for _ in range(2)]
        c, r = kq.KVCache(kq.KQKV_Q8_0, 2, 64, 16, 3, *t), kq.KVRope(kq.KQKV_ROPE_PAIRS, 64, 1e4)
        kq.kqkv_rope_store(c, r, 0, None, 0, None, 0, None, 0, None, 0, None, 0, None, 0)
        kq.kqkv_load(c, 0, None)
        assert kq.kqkv_attn_workspace_bytes(c, 1, 1, 48, 2) >= 0
        kq.kqkv_attn(c, 1, 1, 48, None, None, None, 1, 2, 0, None, 0, 1.0, 0, None, 0)
        return t, c
    assert collected(make)


# ---- what the calls refuse ---------------------------------------------------------
# (each call below gets through the checks of its tensors to a library that records it)

T, B, H, G, D, P, N, S = 3, 2, 2, 2, 32, 16, 5, 4


def i32(*n):
    return Device(torch.zeros(*n, dtype=torch.int32))


def f32(*n):
    return Device(torch.zeros(*n))


def cache(device=0):
    t = [Device(torch.zeros(N * kq.kqkv_page_bytes(kq.KQKV_F16, H, D, P), dtype=torch.uint8), device) for _ in range(2)]
    return kq.KVCache(kq.KQKV_F16, H, D, P, N, *t)


def calls():
    plan = dict(B=B, ctx_len=i32(B), new_len=i32(B), page_tokens=P, table=i32(B, S), table_stride=S, held=i32(B), held_out=i32(B),
                free_pages=i32(N), n_pages=N, n_free=i32(1), n_free_out=i32(1), T=T, slots=i32(T), pos=i32(T), seq_start=i32(B + 1),
                ctx_out=i32(B), err_flag=i32(1))
    store = dict(cache=cache(), rope=kq.KVRope(0, D, 1e4), T=T, pos=i32(1, T), pos_stride=T, slots=i32(T), q_heads=H * G,
                 q=f32(T, H * G * D), ldq=H * G * D, q_out=f32(T, H * G * D), ldq_out=H * G * D, k=f32(T, H * D), ldk=H * D,
                 v=f32(T, H * D), ldv=H * D)
    load = dict(cache=cache(), T=T, slots=i32(T), k=f32(T, H * D), v=f32(T, H * D))
    attn = dict(cache=cache(), B=B, max_q=2, max_ctx=64, ctx_len=i32(B), seq_start=i32(B + 1), table=i32(B, S), table_stride=S,
                q_heads=H * G, T=T, q=f32(T, H * G * D), ldq=H * G * D, scale=0.1, window=0, out=f32(T, H * G * D), ldo=H * G * D,
                workspace=bytes_(1 << 16), workspace_bytes=1 << 16, err_flag=i32(1))
    return dict(kqkv_plan=plan, kqkv_rope_store=store, kqkv_load=load, kqkv_attn=attn)


@pytest.fixture
def library(monkeypatch):
    got = []

    class L:
        def __getattr__(self, fn):
            return lambda *a: got.append((fn, a, binding._torch_c.current)) or 0

    real = binding.lib()
    L.kqkv_page_bytes = staticmethod(real.kqkv_page_bytes)
    monkeypatch.setattr(binding, "_lib", L())
    return got


def tensors_of(kw):
    return [n for n, v in kw.items() if isinstance(v, Device)]


def variants(t):
    """Tensors that are not what `t` is."""
    n = max(t.t.numel(), 2)
    yield Device(t.t.to(torch.int64 if t.dtype == torch.int32 else torch.float64))
    yield Device(t.t.to(torch.int16 if t.dtype == torch.int32 else torch.float16))
    yield Device(t.t.to(torch.float32 if t.dtype == torch.int32 else torch.int32))
    yield Device(t.t, device=1)
    yield Device(t.t, device=None)
    yield Device(torch.zeros(2 * n, dtype=t.dtype)[::2])
    yield Device(torch.zeros(n, n, dtype=t.dtype).t())
    yield Device(torch.zeros(n, 2 * n, dtype=t.dtype)[:, :n])          # rows at another stride than the call says


@pytest.mark.parametrize("fn", ["kqkv_plan", "kqkv_rope_store", "kqkv_load", "kqkv_attn"])
def test_every_tensor_is_checked(library, devices, fn):
    kw = calls()[fn]
    getattr(kq, fn)(**kw)
    assert len(library) == 1 and library[0][1][-1] == 0x7000
    for name in tensors_of(kw):
        for i, bad in enumerate(variants(kw[name])):
            if name == "workspace" and i < 3:                          # bytes of any type
                continue
            with pytest.raises(ValueError):
                getattr(kq, fn)(**dict(kw, **{name: bad}))
            with pytest.raises(ValueError):
                getattr(kq, fn)(**dict(kw, **{name: bad}), stream=5)
    assert len(library) == 1


@pytest.mark.parametrize("fn", ["kqkv_rope_store", "kqkv_load", "kqkv_attn"])
def test_the_cache_is_on_the_tensors_device(library, fn):
    with pytest.raises(ValueError):
        getattr(kq, fn)(**dict(calls()[fn], cache=cache(1)))
    assert not library


def test_a_cache_on_two_devices():
    t = [Device(torch.zeros(N * kq.kqkv_page_bytes(kq.KQKV_F16, H, D, P), dtype=torch.uint8), d) for d in (0, 1)]
    with pytest.raises(ValueError):
        kq.KVCache(kq.KQKV_F16, H, D, P, N, *t)


def test_factors_are_fp32():
    for dtype in (torch.int32, torch.float64, torch.float16):
        with pytest.raises(ValueError):
            kq.KVRope(0, D, 1e4, None, Device(torch.ones(D, dtype=dtype)))


def test_rows_of_wider_buffers(library):
    # q, k and v of one buffer, tables and positions with room, as matrices and by heads
    w = (H * G + 2 * H) * D
    x = torch.zeros(T, w)
    kw = calls()["kqkv_rope_store"]
    kw.update(q=Device(x[:, :H * G * D]), ldq=w, k=Device(x[:, H * G * D:(H * G + H) * D]), ldk=w, v=Device(x[:, (H * G + H) * D:]), ldv=w,
              pos=Device(torch.zeros(3, 9, dtype=torch.int32)[:, :T]), pos_stride=9)
    kq.kqkv_rope_store(**kw)
    kq.kqkv_rope_store(**dict(kw, k=Device(x.view(T, -1, D)[:, H * G:H * G + H])))
    with pytest.raises(ValueError):
        kq.kqkv_rope_store(**dict(kw, k=Device(x.view(T, -1, D)[:, ::2])))
    kw = calls()["kqkv_attn"]
    kq.kqkv_attn(**dict(kw, table=Device(torch.zeros(B, 9, dtype=torch.int32)[:, :S]), table_stride=9))
    assert len(library) == 3


def test_a_call_goes_to_its_tensors_device(library, devices):
    # ... on that device's current stream, or on the one given, whichever device is current
    kw = calls()["kqkv_load"]
    devices.current = 1
    kq.kqkv_load(**kw)
    kq.kqkv_load(**kw, stream=77)
    assert [(a[-1], at) for _, a, at in library] == [(0x7000, 0), (77, 0)]
    # also where the first tensor is an address
    kq.kqkv_load(**dict(kw, slots=0x10000))
    kq.kqkv_load(kw["cache"], T, 0x10000, 0x10000, 0x10000)
    assert [(a[-1], at) for _, a, at in library[2:]] == [(0x7000, 0)] * 2 and devices.current == 1


def test_optional_tensors(library):
    c = calls()
    kq.kqkv_plan(**dict(c["kqkv_plan"], T=0, slots=None, pos=None, err_flag=None))
    kq.kqkv_plan(**dict(c["kqkv_plan"], T=0, slots=None, pos=None))
    kq.kqkv_plan(**dict(c["kqkv_plan"], err_flag=None))
    assert [(not a[13], not a[14], not a[-2]) for _, a, _ in library] == [(True, True, True), (True, True, False), (False, False, True)]
    s = dict(c["kqkv_rope_store"])
    kq.kqkv_rope_store(**dict(s, q=None, q_out=None, q_heads=0))
    kq.kqkv_rope_store(**dict(s, k=None, v=None, slots=None))
    kq.kqkv_load(**dict(c["kqkv_load"], v=None))
    kq.kqkv_attn(**dict(c["kqkv_attn"], workspace=None, workspace_bytes=0, err_flag=None))
    assert len(library) == 7


@pytest.mark.parametrize("fn", ["kqkv_plan", "kqkv_rope_store", "kqkv_load", "kqkv_attn"])
def test_the_first_call_of_a_process(library, devices, monkeypatch, fn):
    load = binding._load_torch
    for name in ("_torch_c", "_int32", "_float32", "_dtype", "_get_device", "_is_contiguous", "_data_ptr"):
        monkeypatch.setattr(binding, name, None)

    def loads():
        load()
        binding._torch_c = devices

    monkeypatch.setattr(binding, "_load_torch", loads)
    kw = calls()[fn]
    getattr(kq, fn)(**kw)
    assert len(library) == 1
