"""ctypes marshalling for libkqgemv.so (see include/kqgemv.h and include/kqkv.h
for semantics)."""
import ctypes
import os

KQ_TYPE_Q4_0, KQ_TYPE_Q8_0, KQ_TYPE_Q2_K, KQ_TYPE_Q3_K = 2, 8, 10, 11
KQ_TYPE_Q4_K, KQ_TYPE_Q5_K, KQ_TYPE_Q6_K = 12, 13, 14
KQKV_F16, KQKV_Q8_0 = 1, 8
KQKV_ROPE_HALVES, KQKV_ROPE_PAIRS = 0, 1

STATUS = {
    0: "KQ_OK", -1: "KQ_ERR_TYPE", -2: "KQ_ERR_SHAPE", -3: "KQ_ERR_M", -4: "KQ_ERR_NULL",
    -5: "KQ_ERR_ALIGN", -6: "KQ_ERR_ARG", -7: "KQ_ERR_LAUNCH", -8: "KQ_ERR_DEVICE",
    -9: "KQ_ERR_IO", -10: "KQ_ERR_FORMAT",
}

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libkqgemv.so")

_lib = None


class GGUFTensor(ctypes.Structure):
    """struct kq_gguf_tensor (include/kqgguf.h)."""
    _fields_ = [("name", ctypes.c_char_p), ("type", ctypes.c_int), ("n_dims", ctypes.c_int),
                ("dims", ctypes.c_int64 * 4), ("offset", ctypes.c_uint64), ("nbytes", ctypes.c_uint64),
                ("data", ctypes.c_void_p)]


class KVCache(ctypes.Structure):
    """struct kqkv_cache (include/kqkv.h).  k and v: contiguous device tensors of
    at least n_pages * kqkv_page_bytes bytes, on one device, or int addresses.  This
    object keeps the tensors alive; when it goes, theirs is any dropped tensor's
    memory, also for calls on other streams that still run."""
    _fields_ = [("type", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("n_pages", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p)]

    def __init__(self, type, kv_heads, head_dim, page_tokens, n_pages, k, v):
        super().__init__(int(type), int(kv_heads), int(head_dim), int(page_tokens), int(n_pages), _addr(k), _addr(v))
        page = lib().kqkv_page_bytes(int(type), int(kv_heads), int(head_dim), int(page_tokens))
        for t in (k, v):
            if t is None or isinstance(t, int) or page < 0:
                continue
            if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < page * int(n_pages):
                raise ValueError("KVCache: k and v must be contiguous device tensors of at least %d bytes" %
                                 (page * int(n_pages)))
        self.device = _device_of("KVCache", (k, v))
        self.tensors = (k, v)


class KVRope(ctypes.Structure):
    """struct kqkv_rope (include/kqkv.h).  sections: the pairs of each axis;
    freq_factors: a tensor (kept alive by this object), an int address or
    None."""
    _fields_ = [("style", ctypes.c_int), ("rot_dims", ctypes.c_int), ("base", ctypes.c_float),
                ("n_axes", ctypes.c_int), ("sections", ctypes.c_int * 4), ("freq_factors", ctypes.c_void_p)]

    def __init__(self, style, rot_dims, base, sections=None, freq_factors=None):
        sections = [int(rot_dims) // 2] if sections is None else [int(n) for n in sections]
        padded = (ctypes.c_int * 4)(*sections[:4])
        super().__init__(int(style), int(rot_dims), float(base), len(sections), padded, _addr(freq_factors))
        if freq_factors is not None and not isinstance(freq_factors, int):
            f = freq_factors
            if not f.is_cuda or not f.is_contiguous() or str(f.dtype) != "torch.float32" or f.numel() < int(rot_dims) // 2:
                raise ValueError("KVRope: freq_factors must be rot_dims / 2 contiguous fp32 values on the device")
        self.device = _device_of("KVRope", (freq_factors,))
        self.tensors = (freq_factors,)


class KQError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (fn, kq_status_string(status), status))


def lib():
    """Load the in-tree shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise ImportError("libkqgemv.so is not built; run __graft_entry__.build() or "
                              "python dequant_gemv_gguf_amd/build.py")
        L = ctypes.CDLL(lib_path)
        P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.kq_version.restype = I
        L.kq_status_string.argtypes = [I]
        L.kq_status_string.restype = ctypes.c_char_p
        L.kq_block_info.argtypes = [I, P, P]
        L.kq_row_bytes.argtypes = [I, I64]
        L.kq_row_bytes.restype = I64
        L.kq_dequant.argtypes = [I, P, I64, P, P]
        L.kq_qgemv.argtypes = [I, P, I64, I64, P, I, P, P]
        L.kq_qgemv_multi.argtypes = [I, P, P, P, I64, P, I, P, P]
        L.kq_qgemv_mc_multi.argtypes = [I, P, P, P, I64, P, I, P, P]
        L.kq_qgemv_mc.argtypes = [I, P, I64, I64, P, I, P, P]
        L.kq_qmoe_workspace_bytes.argtypes = [I, I, I64]
        L.kq_qmoe_workspace_bytes.restype = ctypes.c_size_t
        L.kq_qmoe_gemv.argtypes = [I, P, I64, I64, I64, P, P, I, I, P, I, P, P, P, P]
        L.kq_qmoe_gemv_multi.argtypes = [I, I, P, I64, I64, I64, P, I, I, P, I, P, P, P]
        L.kq_qmoe_gemv_noalloc.argtypes = [I, P, I64, I64, I64, P, P, I, I, P, I, P, P, P]
        U64, CP = ctypes.c_uint64, ctypes.c_char_p
        L.kq_gguf_open.argtypes = [CP, ctypes.POINTER(P)]
        L.kq_gguf_close.argtypes = [P]
        L.kq_gguf_close.restype = None
        L.kq_gguf_version.argtypes = [P]
        L.kq_gguf_alignment.argtypes = [P]
        L.kq_gguf_alignment.restype = I64
        L.kq_gguf_tensor_count.argtypes = [P]
        L.kq_gguf_tensor_count.restype = I64
        L.kq_gguf_find_tensor.argtypes = [P, CP]
        L.kq_gguf_find_tensor.restype = I64
        L.kq_gguf_tensor_info.argtypes = [P, I64, ctypes.POINTER(GGUFTensor)]
        L.kq_gguf_upload.argtypes = [P, I64, P, P]
        L.kq_gguf_meta_count.argtypes = [P]
        L.kq_gguf_meta_count.restype = I64
        L.kq_gguf_meta_key.argtypes = [P, I64, ctypes.POINTER(CP), ctypes.POINTER(I)]
        L.kq_gguf_meta_int.argtypes = [P, CP, ctypes.POINTER(I64)]
        L.kq_gguf_meta_float.argtypes = [P, CP, ctypes.POINTER(ctypes.c_double)]
        L.kq_gguf_meta_string.argtypes = [P, CP, ctypes.POINTER(P), ctypes.POINTER(U64)]
        L.kq_gguf_meta_array.argtypes = [P, CP, ctypes.POINTER(I), ctypes.POINTER(U64), ctypes.POINTER(P)]
        L.kq_gguf_meta_array_string.argtypes = [P, CP, U64, ctypes.POINTER(P), ctypes.POINTER(U64)]
        L.kq_streamer_create.argtypes = [P, ctypes.c_size_t, I, P, ctypes.POINTER(P)]
        L.kq_streamer_destroy.argtypes = [P]
        L.kq_streamer_destroy.restype = None
        L.kq_streamer_sync.argtypes = [P]
        L.kq_stream_qgemv_multi.argtypes = [P, I, P, P, P, I64, P, I, P]
        L.kq_stream_qgemv.argtypes = [P, I, P, I64, I64, P, I, P]
        L.kqkv_page_bytes.argtypes = [I, I, I, I]
        L.kqkv_page_bytes.restype = I64
        L.kqkv_plan.argtypes = [I, P, P, I, P, I64, P, P, P, I64, P, P, I, P, P, P, P, P, P]
        L.kqkv_rope_store.argtypes = [P, P, I, P, I64, P, I, P, I64, P, I64, P, I64, P, I64, P]
        L.kqkv_load.argtypes = [P, I, P, P, P, P]
        L.kqkv_attn_workspace_bytes.argtypes = [P, I, I, I64, I]
        L.kqkv_attn_workspace_bytes.restype = ctypes.c_size_t
        L.kqkv_attn.argtypes = [P, I, I, I64, P, P, P, I64, I, I, P, I64, ctypes.c_float, I, P, I64, P,
                                ctypes.c_size_t, P, P]
        _lib = L
    return _lib


def _ptr(t):
    """Device pointer of a torch tensor, an int address, or None (NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, like):
    if stream is not None:
        return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)
    if like is not None and not isinstance(like, int) and like.is_cuda:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream(like.device).cuda_stream)
    return None


def _check(fn, r):
    if r != 0:
        raise KQError(fn, r)


def kq_version():
    return lib().kq_version()


def kq_status_string(status):
    return lib().kq_status_string(int(status)).decode()


def kq_block_info(qtype):
    qk, nb = ctypes.c_int(), ctypes.c_int()
    _check("kq_block_info", lib().kq_block_info(int(qtype), ctypes.byref(qk), ctypes.byref(nb)))
    return qk.value, nb.value


def kq_row_bytes(qtype, K):
    r = lib().kq_row_bytes(int(qtype), int(K))
    if r < 0:
        raise KQError("kq_row_bytes", int(r))
    return int(r)


def kq_dequant(qtype, src, n_elems, dst, stream=None):
    _check("kq_dequant", lib().kq_dequant(int(qtype), _ptr(src), int(n_elems), _ptr(dst),
                                          _stream(stream, dst)))


def kq_qgemv(qtype, W, N, K, x, M, y, stream=None):
    _check("kq_qgemv", lib().kq_qgemv(int(qtype), _ptr(W), int(N), int(K), _ptr(x), int(M), _ptr(y),
                                      _stream(stream, y)))


def _addr(t):
    if t is None:
        return 0
    return t if isinstance(t, int) else t.data_ptr()


def kq_qgemv_multi(types, Ws, Ns, K, x, M, ys, stream=None):
    """types: one kq_type for every matrix, or a sequence of them; Ws, Ns, ys:
    equal-length sequences (tensors or int addresses, row counts, tensors or
    int addresses), marshalled into the host arrays the C call takes."""
    count = len(Ws)
    if isinstance(types, int):
        types = [types] * count
    if len(types) != count or len(Ns) != count or len(ys) != count:
        raise ValueError("kq_qgemv_multi: types, Ws, Ns and ys must have the same length")
    n = max(count, 1)
    Ta = (ctypes.c_int * n)(*[int(t) for t in types])
    Wa = (ctypes.c_void_p * n)(*[_addr(w) for w in Ws])
    Na = (ctypes.c_int64 * n)(*[int(v) for v in Ns])
    Ya = (ctypes.c_void_p * n)(*[_addr(y) for y in ys])
    like = next((y for y in ys if y is not None and not isinstance(y, int)), None)
    _check("kq_qgemv_multi", lib().kq_qgemv_multi(count, Ta, Wa, Na, int(K), _ptr(x), int(M), Ya,
                                                  _stream(stream, like)))


def kq_qgemv_mc(qtype, W, N, K, x, M, y, stream=None):
    _check("kq_qgemv_mc", lib().kq_qgemv_mc(int(qtype), _ptr(W), int(N), int(K), _ptr(x), int(M), _ptr(y),
                                            _stream(stream, y)))


def kq_qgemv_mc_multi(types, Ws, Ns, K, x, M, ys, stream=None):
    """As kq_qgemv_multi, on the matrix-core kernels."""
    count = len(Ws)
    if isinstance(types, int):
        types = [types] * count
    if len(types) != count or len(Ns) != count or len(ys) != count:
        raise ValueError("kq_qgemv_mc_multi: types, Ws, Ns and ys must have the same length")
    n = max(count, 1)
    Ta = (ctypes.c_int * n)(*[int(t) for t in types])
    Wa = (ctypes.c_void_p * n)(*[_addr(w) for w in Ws])
    Na = (ctypes.c_int64 * n)(*[int(v) for v in Ns])
    Ya = (ctypes.c_void_p * n)(*[_addr(y) for y in ys])
    like = next((y for y in ys if y is not None and not isinstance(y, int)), None)
    _check("kq_qgemv_mc_multi", lib().kq_qgemv_mc_multi(count, Ta, Wa, Na, int(K), _ptr(x), int(M), Ya,
                                                        _stream(stream, like)))


def kq_qmoe_workspace_bytes(T, k, N):
    return int(lib().kq_qmoe_workspace_bytes(int(T), int(k), int(N)))


def kq_qmoe_gemv(qtype, W_exps, E, N, K, ids, route_w, T, k, x, x_mode, y, workspace=None,
                 err_flag=None, stream=None):
    _check("kq_qmoe_gemv", lib().kq_qmoe_gemv(int(qtype), _ptr(W_exps), int(E), int(N), int(K), _ptr(ids),
                                              _ptr(route_w), int(T), int(k), _ptr(x), int(x_mode), _ptr(y),
                                              _ptr(workspace), _ptr(err_flag), _stream(stream, y)))


def kq_qmoe_gemv_noalloc(qtype, W_exps, E, N, K, ids, route_w, T, k, x, x_mode, y, err_flag=None, stream=None):
    _check("kq_qmoe_gemv_noalloc", lib().kq_qmoe_gemv_noalloc(int(qtype), _ptr(W_exps), int(E), int(N), int(K),
                                                              _ptr(ids), _ptr(route_w), int(T), int(k), _ptr(x),
                                                              int(x_mode), _ptr(y), _ptr(err_flag),
                                                              _stream(stream, y)))


def kq_qmoe_gemv_multi(qtype, W_exps, E, N, K, ids, T, k, x, x_mode, ys, err_flag=None, stream=None):
    """W_exps, ys: equal-length sequences (tensors or int addresses) marshalled
    into the host arrays the C call takes."""
    count = len(W_exps)
    if len(ys) != count:
        raise ValueError("kq_qmoe_gemv_multi: W_exps and ys must have the same length")
    n = max(count, 1)
    Wa = (ctypes.c_void_p * n)(*[_addr(w) for w in W_exps])
    Ya = (ctypes.c_void_p * n)(*[_addr(y) for y in ys])
    like = next((y for y in ys if y is not None and not isinstance(y, int)), None)
    _check("kq_qmoe_gemv_multi", lib().kq_qmoe_gemv_multi(count, int(qtype), Wa, int(E), int(N), int(K), _ptr(ids),
                                                          int(T), int(k), _ptr(x), int(x_mode), Ya,
                                                          _ptr(err_flag), _stream(stream, like)))


# ---- GGUF reader (include/kqgguf.h) ------------------------------------------
# A handle is the opaque kq_gguf* as an int.

def kq_gguf_open(path):
    h = ctypes.c_void_p()
    _check("kq_gguf_open", lib().kq_gguf_open(os.fsencode(path), ctypes.byref(h)))
    return h.value


def kq_gguf_close(h):
    lib().kq_gguf_close(h)


def kq_gguf_version(h):
    return int(lib().kq_gguf_version(h))


def kq_gguf_alignment(h):
    return int(lib().kq_gguf_alignment(h))


def kq_gguf_tensor_count(h):
    return int(lib().kq_gguf_tensor_count(h))


def kq_gguf_find_tensor(h, name):
    r = int(lib().kq_gguf_find_tensor(h, name.encode()))
    if r < 0:
        raise KQError("kq_gguf_find_tensor", r)
    return r


def kq_gguf_tensor_info(h, i):
    t = GGUFTensor()
    _check("kq_gguf_tensor_info", lib().kq_gguf_tensor_info(h, int(i), ctypes.byref(t)))
    return {"name": t.name.decode(), "type": t.type, "n_dims": t.n_dims, "dims": tuple(t.dims[:t.n_dims]),
            "offset": int(t.offset), "nbytes": int(t.nbytes), "data": t.data}


def kq_gguf_upload(h, i, dst, stream=None):
    _check("kq_gguf_upload", lib().kq_gguf_upload(h, int(i), _ptr(dst), _stream(stream, dst)))


def kq_gguf_meta_count(h):
    return int(lib().kq_gguf_meta_count(h))


def kq_gguf_meta_key(h, i):
    k, t = ctypes.c_char_p(), ctypes.c_int()
    _check("kq_gguf_meta_key", lib().kq_gguf_meta_key(h, int(i), ctypes.byref(k), ctypes.byref(t)))
    return k.value.decode(), t.value


def kq_gguf_meta_int(h, key):
    v = ctypes.c_int64()
    _check("kq_gguf_meta_int", lib().kq_gguf_meta_int(h, key.encode(), ctypes.byref(v)))
    return v.value


def kq_gguf_meta_float(h, key):
    v = ctypes.c_double()
    _check("kq_gguf_meta_float", lib().kq_gguf_meta_float(h, key.encode(), ctypes.byref(v)))
    return v.value


def kq_gguf_meta_string(h, key):
    p, n = ctypes.c_void_p(), ctypes.c_uint64()
    _check("kq_gguf_meta_string", lib().kq_gguf_meta_string(h, key.encode(), ctypes.byref(p), ctypes.byref(n)))
    return ctypes.string_at(p.value, n.value) if n.value else b""


def kq_gguf_meta_array(h, key):
    """(element type, count, host address of the packed elements or None)."""
    t, n, p = ctypes.c_int(), ctypes.c_uint64(), ctypes.c_void_p()
    _check("kq_gguf_meta_array", lib().kq_gguf_meta_array(h, key.encode(), ctypes.byref(t), ctypes.byref(n),
                                                          ctypes.byref(p)))
    return t.value, n.value, p.value


def kq_gguf_meta_array_string(h, key, j):
    p, n = ctypes.c_void_p(), ctypes.c_uint64()
    _check("kq_gguf_meta_array_string", lib().kq_gguf_meta_array_string(h, key.encode(), int(j), ctypes.byref(p),
                                                                        ctypes.byref(n)))
    return ctypes.string_at(p.value, n.value) if n.value else b""


# ---- host-streamed GEMV (include/kqstream.h) -----------------------------------
# A streamer is the opaque kq_streamer* as an int.  Weights are HOST tensors or
# addresses (page-locked for overlap); x and y are device tensors.

def kq_streamer_create(slots, slot_bytes, nslots, stream=None):
    h = ctypes.c_void_p()
    _check("kq_streamer_create", lib().kq_streamer_create(_ptr(slots), int(slot_bytes), int(nslots),
                                                          _stream(stream, slots), ctypes.byref(h)))
    return h.value


def kq_streamer_destroy(h):
    lib().kq_streamer_destroy(h)


def kq_streamer_sync(h):
    _check("kq_streamer_sync", lib().kq_streamer_sync(h))


def kq_stream_qgemv_multi(h, types, Ws, Ns, K, x, M, ys):
    count = len(Ws)
    if isinstance(types, int):
        types = [types] * count
    if len(types) != count or len(Ns) != count or len(ys) != count:
        raise ValueError("kq_stream_qgemv_multi: types, Ws, Ns and ys must have the same length")
    n = max(count, 1)
    Ta = (ctypes.c_int * n)(*[int(t) for t in types])
    Wa = (ctypes.c_void_p * n)(*[_addr(w) for w in Ws])
    Na = (ctypes.c_int64 * n)(*[int(v) for v in Ns])
    Ya = (ctypes.c_void_p * n)(*[_addr(y) for y in ys])
    _check("kq_stream_qgemv_multi", lib().kq_stream_qgemv_multi(h, count, Ta, Wa, Na, int(K), _ptr(x), int(M), Ya))


def kq_stream_qgemv(h, qtype, W, N, K, x, M, y):
    _check("kq_stream_qgemv", lib().kq_stream_qgemv(h, int(qtype), _ptr(W), int(N), int(K), _ptr(x), int(M),
                                                    _ptr(y)))


# ---- paged key-value cache (include/kqkv.h) -------------------------------------
# cache: a KVCache, rope: a KVRope (or None).  Tensors or int addresses.  A call
# goes to the device that its tensors are on, on that device's current stream
# where none is given.  Tensors are checked for what they are, not for their
# sizes: all on one device, int32 or fp32 as the header says, contiguous, or with
# rows that are, as far apart as the call's stride says.

# These calls are made once per layer and token, and take a few microseconds on
# the GPU: what the host spends on them shows.  So the current stream is asked
# for by torch._C's raw calls (0.1 us; torch.cuda.current_stream makes a Stream
# object, 2.8 us), addresses go to ctypes as ints, and a call's tensors are
# looked over together, one property after the other (1.1 to 1.7 us a call).

_torch_c = _int32 = _float32 = _dtype = _get_device = _is_contiguous = _data_ptr = None      # until a tensor comes


def _struct(s):
    """A KVCache or KVRope as an argument.  (Made for each call: a byref that the
    object itself held would be a cycle that is never collected, and keep the
    buffers.)"""
    return None if s is None else ctypes.byref(s)


def _load_torch():
    global _torch_c, _int32, _float32, _dtype, _get_device, _is_contiguous, _data_ptr
    import torch
    T = torch.Tensor
    _int32, _float32 = torch.int32, torch.float32
    _dtype, _get_device, _is_contiguous, _data_ptr = T.dtype.__get__, T.get_device, T.is_contiguous, T.data_ptr
    _torch_c = torch._C


def _device_of(fn, tensors):
    """The device index of the tensors among `tensors` (None where there are none)."""
    device = None
    for t in tensors:
        if t is None or isinstance(t, int):
            continue
        if not t.is_cuda:
            raise ValueError("%s: tensors must be on the device" % fn)
        if device is None:
            device = t.get_device()
        elif t.get_device() != device:
            raise ValueError("%s: tensors on devices %d and %d" % (fn, device, t.get_device()))
    return device


def _rows_apart(t, ld):
    """Whether t[i] are contiguous and ld elements apart."""
    shape, strides, n = t.shape, t.stride(), 1
    for size, stride in zip(reversed(shape[1:]), reversed(strides[1:])):
        if size != 1 and stride != n:
            return False
        n *= size
    return len(shape) > 1 and (shape[0] == 1 or strides[0] == ld)


def _addresses(fn, device, dtypes, tensors, strides):
    """The tensors' addresses (int addresses and None as they are), all on this
    device and of these dtypes (those behind the last one's: of any).  strides:
    the rows' of those that have any, else None."""
    n = len(tensors)
    try:
        if (list(map(_get_device, tensors)).count(device) == n and list(map(_is_contiguous, tensors)).count(True) == n and
                list(map(_dtype, tensors))[:len(dtypes)] == dtypes):
            return list(map(_data_ptr, tensors))
    except TypeError:                                  # not all are tensors
        pass
    out = []
    for i, t in enumerate(tensors):
        if t is not None and not isinstance(t, int):
            if _device_of(fn, (t,)) != device:
                raise ValueError("%s: tensors on devices %d and %d" % (fn, device, t.get_device()))
            if i < len(dtypes) and t.dtype != dtypes[i]:
                raise ValueError("%s: a %s tensor where %s is asked for" % (fn, t.dtype, dtypes[i]))
            if not t.is_contiguous() and (strides[i] is None or not _rows_apart(t, strides[i])):
                raise ValueError("%s: a tensor of shape %s and strides %s is neither contiguous nor rows at the call's stride"
                                 % (fn, tuple(t.shape), t.stride()))
        out.append(_addr(t))
    return out


def _target(fn, stream, first, others, *structs):
    """Where a call goes: the device of its tensors (`first` mostly is one) or of
    its cache, which has to be the same (None: the current one), and the stream."""
    if first is not None and type(first) is not int:
        device = first.get_device()
        if device < 0:
            raise ValueError("%s: tensors must be on the device" % fn)
    else:
        device = _device_of(fn, others)
    for s in structs:
        if s is not None and s.device != device and s.device is not None:
            if device is not None:
                raise ValueError("%s: tensors on devices %d and %d" % (fn, device, s.device))
            device = s.device
    if device is not None:
        if _torch_c is None:
            _load_torch()
        if stream is None:
            stream = _torch_c._cuda_getCurrentRawStream(device)
    if stream is not None and type(stream) is not int:
        stream = stream.cuda_stream
    return device, stream


def _call(fn, f, device, args):
    """f(*args) with `device` current."""
    if device is None or device == _torch_c._cuda_getDevice():
        r = f(*args)
    else:
        import torch
        with torch.cuda.device(device):
            r = f(*args)
    if r:
        raise KQError(fn, r)


def kqkv_page_bytes(qtype, kv_heads, head_dim, page_tokens):
    r = int(lib().kqkv_page_bytes(int(qtype), int(kv_heads), int(head_dim), int(page_tokens)))
    if r < 0:
        raise KQError("kqkv_page_bytes", r)
    return r


def kqkv_plan(B, ctx_len, new_len, page_tokens, table, table_stride, held, held_out, free_pages, n_pages, n_free,
              n_free_out, T, slots, pos, seq_start, ctx_out, err_flag=None, stream=None):
    if slots is None and pos is None and err_flag is None:
        tensors = (ctx_len, new_len, held, held_out, free_pages, n_free, n_free_out, seq_start, ctx_out, table)
    elif err_flag is None:
        tensors = (ctx_len, new_len, held, held_out, free_pages, n_free, n_free_out, seq_start, ctx_out, table, slots, pos)
    else:
        tensors = (ctx_len, new_len, held, held_out, free_pages, n_free, n_free_out, seq_start, ctx_out, table, slots, pos,
                   err_flag)
    device, stream = _target("kqkv_plan", stream, ctx_len, tensors)
    a = _addresses("kqkv_plan", device, [_int32] * len(tensors), tensors,
                   (None, None, None, None, None, None, None, None, None, table_stride, None, None, None))
    a += [None] * (13 - len(a))
    _call("kqkv_plan", (_lib or lib()).kqkv_plan, device,
          (B, a[0], a[1], page_tokens, a[9], table_stride, a[2], a[3], a[4], n_pages, a[5], a[6], T, a[10], a[11], a[7],
           a[8], a[12], stream))


def kqkv_rope_store(cache, rope, T, pos, pos_stride, slots, q_heads, q, ldq, q_out, ldq_out, k, ldk, v, ldv,
                    stream=None):
    fn = "kqkv_rope_store"
    if q is None and q_out is None:
        tensors, strides = (pos, slots, k, v), (pos_stride, None, ldk, ldv)
    else:
        tensors, strides = (pos, slots, k, v, q, q_out), (pos_stride, None, ldk, ldv, ldq, ldq_out)
    device, stream = _target(fn, stream, slots, tensors, cache, rope)
    a = _addresses(fn, device, [_int32, _int32, _float32, _float32, _float32, _float32][:len(tensors)], tensors, strides)
    if len(a) == 4:
        a += (None, None)
    _call(fn, (_lib or lib()).kqkv_rope_store, device,
          (_struct(cache), _struct(rope), T, a[0], pos_stride, a[1], q_heads, a[4], ldq, a[5], ldq_out, a[2], ldk, a[3],
           ldv, stream))


def kqkv_load(cache, T, slots, k=None, v=None, stream=None):
    device, stream = _target("kqkv_load", stream, slots, (k, v), cache)
    a = _addresses("kqkv_load", device, [_int32, _float32, _float32], (slots, k, v), (None, None, None))
    _call("kqkv_load", (_lib or lib()).kqkv_load, device, (_struct(cache), T, a[0], a[1], a[2], stream))


def kqkv_attn_workspace_bytes(cache, B, max_q, max_ctx, q_heads):
    return int(lib().kqkv_attn_workspace_bytes(_struct(cache), int(B), int(max_q), int(max_ctx), int(q_heads)))


def kqkv_attn(cache, B, max_q, max_ctx, ctx_len, seq_start, table, table_stride, q_heads, T, q, ldq, scale, window,
              out, ldo, workspace=None, workspace_bytes=0, err_flag=None, stream=None):
    fn = "kqkv_attn"
    tensors = (ctx_len, seq_start, table, q, out) if err_flag is None else (ctx_len, seq_start, table, q, out, err_flag)
    typed = len(tensors)
    if workspace is not None:
        tensors += (workspace,)
    device, stream = _target(fn, stream, q, tensors, cache)
    types = [_int32, _int32, _int32, _float32, _float32, _int32][:typed]
    a = _addresses(fn, device, types, tensors, (None, None, table_stride, ldq, ldo, None, None))
    _call(fn, (_lib or lib()).kqkv_attn, device,
          (_struct(cache), B, max_q, max_ctx, a[0], a[1], a[2], table_stride, q_heads, T, a[3], ldq, scale, window, a[4],
           ldo, a[-1] if workspace is not None else None, workspace_bytes, a[5] if err_flag is not None else None, stream))
