"""CPU checks of the paged-cache binding with stand-ins for device tensors:
what it keeps alive, and what it refuses before the library is called."""
import gc
import weakref

import pytest

import dequant_gemv_gguf_amd as kq

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
        return self.device

    def data_ptr(self):
        return self.at


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
