"""Python binding of the tq2-gb300 C ABI (``include/tq2.h``).

Argument marshalling only: every function forwards device pointers, sizes
and the current CUDA stream of torch to the shared library
``libtq2gb300.so`` built from ``csrc/``.  There is no fallback: if the
library is missing or fails to load, every call raises.

Tensors must live on the current CUDA device, be contiguous and have the
dtype the C ABI states (float32 for activations and outputs, uint8 / int16
bit patterns for packed data).  The ``q4_``, ``moe_`` and ``kv8_`` calls also take
float16 and bfloat16 activations, and rows with a stride.
"""
import ctypes
import os

__all__ = [
    "load", "lib_path", "TQ2Error", "Weight", "tq2_upload", "tq2_gemm", "tq2_gemm_path", "tq2_gemm_tensor_tuned",
    "tq2_gemm_skinny_static", "tq2_gemm_grouped", "GroupedGemv", "tq2_unpack", "tq2_dequant_f16", "tq2_quantize", "blr_expand_bits", "blr_forward", "blr_backward", "blr_forward_paths", "blr_backward_paths", "blr_sign_grads",
    "Q4Weight", "q4_upload", "q4_dequant", "q4_quantize", "q4_gemm", "moe_route", "moe_route_backward", "moe_experts",
    "KV8Cache", "KV8Batch", "kv8_write", "kv8_read", "kv8_attention",
    "device_status", "release_scratch", "debug_wait_timeout", "PATH_AUTO", "PATH_SKINNY", "PATH_TENSOR",
]

PATH_AUTO, PATH_SKINNY, PATH_TENSOR = 0, 1, 2
_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libtq2gb300.so")
_lib = None

_P, _I64, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_SIGS = {
    "tq2_status_string": (ctypes.c_char_p, [_I]),
    "tq2_last_error": (ctypes.c_char_p, []),
    "tq2_version": (ctypes.c_char_p, []),
    "tq2_device_status": (_I, [_P]),
    "tq2_release_scratch": (_I, []),
    "tq2_debug_wait_timeout": (_I, [ctypes.c_uint64, _P]),
    "tq2_upload": (_I, [_P, _I64, _I64, ctypes.POINTER(_P), _P]),
    "tq2_free": (_I, [_P]),
    "tq2_shape": (_I, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "tq2_gemm": (_I, [_P, _P, _P, _I64, _I64, _I64, _P]),
    "tq2_gemm_path": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P]),
    "tq2_gemm_tensor_tuned": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _I, _P]),
    "tq2_gemm_skinny_static": (_I, [_P, _P, _P, _I64, _I64, _I64, _P]),
    "tq2_gemm_grouped": (_I, [_P, _P, _P, _I, _I64, _I64, _P]),
    "tq2_unpack": (_I, [_P, _P, _P]),
    "tq2_dequant_f16": (_I, [_P, _P, _P]),
    "tq2_quantize": (_I, [_P, _I64, _I64, _P, _P]),
    "blr_expand_bits": (_I, [_P, _I64, _I64, _P, _I, _P]),
    "blr_forward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P]),
    "blr_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                          _I64, _I64, _I64, _I64, _F, _P]),
    "blr_forward_paths": (_I, [_P, _I, _P, _P, _I64, _I64, _I64, _I64, _P]),
    "blr_backward_paths": (_I, [_P, _I, _P, _P, _P, _I64, _I64, _I64, _I64, _F, _P]),
    "blr_sign_grads": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _F, _P]),
    "q4_upload": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, ctypes.POINTER(_P), _P]),
    "q4_free": (_I, [_P]),
    "q4_shape": (_I, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I)]),
    "q4_dequant": (_I, [_P, _P, _P]),
    "q4_quantize": (_I, [_P, _I, _I64, _I64, _I, _P, _P, _P, _P]),
    "q4_gemm": (_I, [_P, _P, _I64, _P, _I64, _I, _I64, _P]),
    "moe_route": (_I, [_P, _I64, _I, _P, _I64, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P]),
    "moe_route_backward": (_I, [_P, _I64, _I, _P, _P, _P, _P, _I64, _I64, _I, _I, _I, _I, _F, _P]),
    "moe_experts": (_I, [_P, _P, _P, _P, _I64, _I, _P, _P, _P, _P, _P, _I64, _I64, _I, _P]),
    "kv8_write": (_I, [_P, _P, _P, _I64, _I64, _P, _I64, _I64, _I, _I64, _P]),
    "kv8_read": (_I, [_P, _P, _P, _I64, _I64, _P, _I64, _I64, _I, _I64, _P]),
    "kv8_attention": (_I, [_P, _P, _P, _I64, _I64, _P, _I64, _I64, _I, _P, _I64, _I, _F, _I, _I64, _I64, _P]),
}


class BlrPath(ctypes.Structure):
    """``blr_path`` of include/tq2.h: device pointers of one path."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("bits_u", "bits_v", "h", "l", "g", "a_save", "c_save", "dh", "dl", "dg")]


class _Kv8Cache(ctypes.Structure):
    """``kv8_cache`` of include/tq2.h."""
    _fields_ = [("codes", _P), ("scales", _P), ("blocks", _I64), ("heads", _I), ("tokens", _I), ("dim", _I)]


class _Kv8Batch(ctypes.Structure):
    """``kv8_batch`` of include/tq2.h."""
    _fields_ = [("table", _P), ("ld", _I64), ("offsets", _P), ("lens", _P), ("width", _I), ("seqs", _I)]


class TQ2Error(RuntimeError):
    def __init__(self, status, where):
        msg = load().tq2_last_error().decode(errors="replace")
        name = load().tq2_status_string(status).decode()
        super().__init__(f"{where}: {name} ({status}): {msg}")
        self.status = status


def load():
    """Load the shared library (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(f"{lib_path} is missing; build it with binary_packed_weight_gb300.build.build()")
        lib = ctypes.CDLL(lib_path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def _check(status, where):
    if status != 0:
        raise TQ2Error(status, where)


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class Weight:
    """A ``BlockTQ2_0_g128`` weight resident on the GPU (owns a C handle)."""

    def __init__(self, handle, N, K):
        self._h, self.N, self.K = handle, N, K

    @property
    def handle(self):
        return self._h

    def free(self):
        if self._h:
            h, self._h = self._h, None                     # taken back even where an error is reported
            _check(load().tq2_free(h), "tq2_free")

    def __del__(self):
        try:
            if self._h and _lib is not None:
                _lib.tq2_free(self._h)
        except Exception:
            pass


def tq2_upload(aos, N, K, stream=None):
    """Upload AoS block bytes (host ``bytes`` / numpy uint8) -> :class:`Weight`."""
    buf = bytes(aos) if not isinstance(aos, (bytes, bytearray)) else aos
    arr = (ctypes.c_uint8 * len(buf)).from_buffer_copy(buf)
    h = ctypes.c_void_p()
    _check(load().tq2_upload(ctypes.cast(arr, _P), N, K, ctypes.byref(h), _stream(stream)), "tq2_upload")
    return Weight(h.value, N, K)


def tq2_gemm(w, x, out, stream=None):
    M, K = x.shape
    _check(load().tq2_gemm(w.handle, _ptr(x), _ptr(out), M, w.N, K, _stream(stream)), "tq2_gemm")
    return out


def tq2_gemm_path(w, x, out, path, stream=None):
    M, K = x.shape
    _check(load().tq2_gemm_path(w.handle, _ptr(x), _ptr(out), M, w.N, K, path, _stream(stream)), "tq2_gemm_path")
    return out


def tq2_gemm_tensor_tuned(w, x, out, bn=0, splits=0, stream=None):
    """The tensor-core path with a chosen token tile (bn) and K-split count."""
    M, K = x.shape
    _check(load().tq2_gemm_tensor_tuned(w.handle, _ptr(x), _ptr(out), M, w.N, K, int(bn), int(splits),
                                        _stream(stream)), "tq2_gemm_tensor_tuned")
    return out


def tq2_gemm_skinny_static(w, x, out, stream=None):
    """Skinny GEMM (M <= 16) that allocates nothing: its scratch is a fixed
    device array inside the library (see include/tq2.h)."""
    M, K = x.shape
    _check(load().tq2_gemm_skinny_static(w.handle, _ptr(x), _ptr(out), M, w.N, K, _stream(stream)),
           "tq2_gemm_skinny_static")
    return out


def tq2_gemm_grouped(ws, xs, outs, stream=None):
    """G independent GEMVs (M <= 8, same K) in one launch: outs[g] = xs[g] @ W_g^T."""
    G = len(ws)
    M, K = xs[0].shape
    hs = (_P * G)(*[w.handle for w in ws])
    xp = (_P * G)(*[x.data_ptr() for x in xs])
    op = (_P * G)(*[o.data_ptr() for o in outs])
    _check(load().tq2_gemm_grouped(ctypes.cast(hs, _P), ctypes.cast(xp, _P), ctypes.cast(op, _P), G, M, K,
                                   _stream(stream)), "tq2_gemm_grouped")
    return outs


class GroupedGemv:
    """tq2_gemm_grouped with its arguments marshalled once: the handle and
    pointer arrays are built at construction (the tensors are kept alive), so a
    loop that calls the same group every step pays one C call per step."""

    def __init__(self, ws, xs, outs):
        self._keep = (list(ws), list(xs), list(outs))
        self.G = len(ws)
        self.M, self.K = xs[0].shape
        self._hs = (_P * self.G)(*[w.handle for w in ws])
        self._xp = (_P * self.G)(*[x.data_ptr() for x in xs])
        self._op = (_P * self.G)(*[o.data_ptr() for o in outs])
        self._args = (ctypes.cast(self._hs, _P), ctypes.cast(self._xp, _P), ctypes.cast(self._op, _P))

    def __call__(self, stream=None):
        _check(load().tq2_gemm_grouped(*self._args, self.G, self.M, self.K, _stream(stream)), "tq2_gemm_grouped")
        return self._keep[2]


def tq2_unpack(w, stream=None):
    n = w.N * (w.K // 128) * 34
    buf = (ctypes.c_uint8 * n)()
    _check(load().tq2_unpack(w.handle, ctypes.cast(buf, _P), _stream(stream)), "tq2_unpack")
    return bytes(buf)


def tq2_dequant_f16(w, out_u16, stream=None):
    _check(load().tq2_dequant_f16(w.handle, _ptr(out_u16), _stream(stream)), "tq2_dequant_f16")
    return out_u16


def tq2_quantize(w, aos_out, stream=None):
    """f32 weights ``w`` [N, K] (device) -> BlockTQ2_0_g128 blocks in ``aos_out``
    (device uint8, N*(K/128)*34 bytes)."""
    N, K = w.shape
    _check(load().tq2_quantize(_ptr(w), N, K, _ptr(aos_out), _stream(stream)), "tq2_quantize")
    return aos_out


def blr_expand_bits(bits, rows, r, plane, transpose, stream=None):
    _check(load().blr_expand_bits(_ptr(bits), rows, r, _ptr(plane), int(transpose), _stream(stream)),
           "blr_expand_bits")
    return plane


def blr_forward(bits_u, bits_v, h, l, g, x, y, a_save, c_save=None, stream=None):
    T, d_in = x.shape
    d_out, r = h.numel(), l.numel()
    _check(load().blr_forward(_ptr(bits_u), _ptr(bits_v), _ptr(h), _ptr(l), _ptr(g), _ptr(x), _ptr(y),
                              _ptr(a_save), _ptr(c_save), T, d_in, d_out, r, _stream(stream)), "blr_forward")
    return y


def blr_backward(bits_u, bits_v, h, l, g, x, dy, a_save, c_save, dx, dh, dl, dg, gscale=1.0, stream=None):
    T, d_in = x.shape
    d_out, r = h.numel(), l.numel()
    _check(load().blr_backward(_ptr(bits_u), _ptr(bits_v), _ptr(h), _ptr(l), _ptr(g), _ptr(x), _ptr(dy),
                               _ptr(a_save), _ptr(c_save), _ptr(dx), _ptr(dh), _ptr(dl), _ptr(dg),
                               T, d_in, d_out, r, float(gscale), _stream(stream)), "blr_backward")
    return dx


def _paths_array(paths):
    """List of dicts of tensors (keys as BlrPath's fields; missing ones are NULL)."""
    arr = (BlrPath * len(paths))()
    for i, p in enumerate(paths):
        for name, _ in BlrPath._fields_:
            setattr(arr[i], name, _ptr(p.get(name)))
    return arr


def blr_forward_paths(paths, x, y, stream=None):
    """y = sum over paths, combined with the pages' rounding (see include/tq2.h)."""
    T, d_in = x.shape
    d_out, r = paths[0]["h"].numel(), paths[0]["l"].numel()
    arr = _paths_array(paths)
    _check(load().blr_forward_paths(ctypes.cast(arr, _P), len(paths), _ptr(x), _ptr(y), T, d_in, d_out, r,
                                    _stream(stream)), "blr_forward_paths")
    return y


def blr_backward_paths(paths, x, dy, dx, gscale=1.0, stream=None):
    T, d_in = x.shape
    d_out, r = paths[0]["h"].numel(), paths[0]["l"].numel()
    arr = _paths_array(paths)
    _check(load().blr_backward_paths(ctypes.cast(arr, _P), len(paths), _ptr(x), _ptr(dy), _ptr(dx), T, d_in, d_out,
                                     r, float(gscale), _stream(stream)), "blr_backward_paths")
    return dx


def blr_sign_grads(bits_u, h, l, g, x, dy, a_save, gu, gv, gscale=1.0, stream=None):
    """G_U [d_out, r] and G_V [d_in, r] of one path (see include/tq2.h)."""
    T, d_in = x.shape
    d_out, r = h.numel(), l.numel()
    _check(load().blr_sign_grads(_ptr(bits_u), _ptr(h), _ptr(l), _ptr(g), _ptr(x), _ptr(dy), _ptr(a_save), _ptr(gu),
                                 _ptr(gv), T, d_in, d_out, r, float(gscale), _stream(stream)), "blr_sign_grads")
    return gu, gv


class Q4Weight:
    """E 4-bit matrices [N, K] with group scales resident on the GPU (owns a C handle)."""

    def __init__(self, handle, E, N, K, group):
        self._h, self.E, self.N, self.K, self.group = handle, E, N, K, group

    @property
    def handle(self):
        return self._h

    def free(self):
        if self._h:
            h, self._h = self._h, None                     # taken back even where an error is reported
            _check(load().q4_free(h), "q4_free")

    def __del__(self):
        try:
            if self._h and _lib is not None:
                _lib.q4_free(self._h)
        except Exception:
            pass


_dtypes = {}
_names = {}
_raw_stream = None


def _torch_names():
    """torch objects the argument checks compare with (torch is imported on first use)."""
    import torch
    _dtypes.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    _names.update({"int32": torch.int32, "uint8": torch.uint8, "float32": torch.float32, "float16": torch.float16})


def _dtype(t, where):
    """tq2_dtype of a tensor."""
    if not _dtypes:
        _torch_names()
    d = _dtypes.get(t.dtype)
    if d is None:
        raise TypeError(f"{where}: dtype {t.dtype} is not float32, float16 or bfloat16")
    return d


def _rows(t, rows, cols, where, name):
    """Row stride of a [rows, cols] tensor whose rows are contiguous."""
    if t.shape != (rows, cols):
        raise ValueError(f"{where}: {name} must be [{rows}, {cols}], got {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{where}: {name} must be on the GPU")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{where}: the rows of {name} must be contiguous")
    return ld if rows > 1 else max(ld, cols)               # (a lone row's stride says nothing)


def _plane(t, shape, dtype, where, name, host=False):
    """The address of a dense tensor of a given shape and dtype (a torch dtype's name); host: a CPU one will do."""
    if not _names:
        _torch_names()
    if t.dtype is not _names[dtype] or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if not (t.is_cuda or host):
        raise ValueError(f"{where}: {name} must be on the GPU")
    return t.data_ptr()


def _on(t, stream):
    """The stream of a call on tensor ``t``: the given one or torch's current one of its device."""
    if stream is not None:
        return int(stream)
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = torch._C._cuda_getCurrentRawStream
    return _raw_stream(t.get_device())


def _group(group, where):
    """A group size by which K can be divided (which ones there are the library says)."""
    if group < 1:
        raise ValueError(f"{where}: group must be 32, 64 or 128, got {group}")
    return group


def q4_upload(codes, scales, zeros=None, group=128, stream=None):
    """4-bit weights -> :class:`Q4Weight`.  ``codes`` uint8 [E, N, K/2] or [N, K/2] (even k in the low
    half byte), ``scales`` float16 and ``zeros`` uint8 (or None: 8) [.., N, K/group]; CPU or CUDA tensors."""
    shape = tuple(codes.shape) if codes.dim() == 3 else (1,) + tuple(codes.shape)
    if len(shape) != 3:
        raise ValueError(f"q4_upload: codes must be [E, N, K/2] or [N, K/2], got {list(codes.shape)}")
    E, N, K = shape[0], shape[1], 2 * shape[2]
    _group(group, "q4_upload")
    lead = tuple(codes.shape)[:-1]
    _plane(codes, lead + (K // 2,), "uint8", "q4_upload", "codes", host=True)
    _plane(scales, lead + (K // group,), "float16", "q4_upload", "scales", host=True)
    if zeros is not None:
        _plane(zeros, lead + (K // group,), "uint8", "q4_upload", "zeros", host=True)
    h = ctypes.c_void_p()
    _check(load().q4_upload(_ptr(codes), _ptr(scales), _ptr(zeros), E, N, K, group, ctypes.byref(h),
                            _stream(stream)), "q4_upload")
    return Q4Weight(h.value, E, N, K, group)


def q4_dequant(w, out, stream=None):
    """W as float32 [E, N, K] (exact)."""
    if out.numel() != w.E * w.N * w.K or not (out.is_contiguous() and out.is_cuda) or str(out.dtype) != "torch.float32":
        raise ValueError(f"q4_dequant: out must be contiguous float32 on the GPU, of {w.E}*{w.N}*{w.K} elements")
    _check(load().q4_dequant(w.handle, _ptr(out), _stream(stream)), "q4_dequant")
    return out


def q4_quantize(w, codes, scales, zeros=None, group=128, stream=None):
    """Plain weights [.., N, K] to the planes :func:`q4_upload` takes (see include/tq2.h)."""
    if w.dim() < 1:
        raise ValueError("q4_quantize: w must have rows of K weights, got a scalar")
    K = w.shape[-1]
    _group(group, "q4_quantize")
    lead = tuple(w.shape)[:-1]
    if not (w.is_contiguous() and w.is_cuda):
        raise ValueError("q4_quantize: w must be contiguous and on the GPU")
    _plane(codes, lead + (K // 2,), "uint8", "q4_quantize", "codes")
    _plane(scales, lead + (K // group,), "float16", "q4_quantize", "scales")
    if zeros is not None:
        _plane(zeros, lead + (K // group,), "uint8", "q4_quantize", "zeros")
    _check(load().q4_quantize(_ptr(w), _dtype(w, "q4_quantize"), w.numel() // max(K, 1), K, group, _ptr(codes),
                              _ptr(scales), _ptr(zeros), _stream(stream)), "q4_quantize")
    return codes, scales, zeros


def q4_gemm(w, x, out, stream=None):
    """out [M, N] = x [M, K] @ W^T for a weight with one matrix; rows may be strided."""
    M = x.shape[0]
    if out.dtype is not x.dtype:
        raise TypeError("q4_gemm: x and out must have the same dtype")
    _check((_lib or load()).q4_gemm(w._h, x.data_ptr(), _rows(x, M, w.K, "q4_gemm", "x"), out.data_ptr(),
                                    _rows(out, M, w.N, "q4_gemm", "out"), _dtype(x, "q4_gemm"), M, _on(x, stream)),
           "q4_gemm")
    return out


_SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score, where):
    try:
        return _SCORES[score]
    except KeyError:
        raise ValueError(f"{where}: score must be one of {sorted(_SCORES)}, got {score!r}") from None


def moe_route(logits, ids, weights, offsets=None, slots=None, bias=None, score="softmax", groups=1, top_groups=1,
              renorm=True, scale=1.0, stream=None):
    """Selection, weights and plan of a router (see include/tq2.h): ``logits`` [T, E] -> ``ids`` int32 and
    ``weights`` float32 [T, k], and unless None ``offsets`` int32 [E+1], ``slots`` int32 [T*k]."""
    T, E = logits.shape
    k = ids.shape[1]
    at = "moe_route"
    _check((_lib or load()).moe_route(
        logits.data_ptr(), _rows(logits, T, E, at, "logits"), _dtype(logits, at),
        None if bias is None else _plane(bias, (E,), "float32", at, "bias"), T, E, k, _score(score, at), groups,
        top_groups, 1 if renorm else 0, scale, _plane(ids, (T, k), "int32", at, "ids"),
        _plane(weights, (T, k), "float32", at, "weights"),
        None if offsets is None else _plane(offsets, (E + 1,), "int32", at, "offsets"),
        None if slots is None else _plane(slots, (T * k,), "int32", at, "slots"), _on(logits, stream)), at)
    return ids, weights, offsets, slots


def moe_route_backward(logits, ids, dweights, dlogits, bias=None, score="softmax", renorm=True, scale=1.0,
                       stream=None):
    """Gradient of :func:`moe_route`'s weights to its logits, ``dlogits`` [T, E] in the logits' dtype."""
    T, E = logits.shape
    k = ids.shape[1]
    at = "moe_route_backward"
    if dlogits.dtype is not logits.dtype:
        raise TypeError("moe_route_backward: logits and dlogits must have the same dtype")
    _check((_lib or load()).moe_route_backward(
        logits.data_ptr(), _rows(logits, T, E, at, "logits"), _dtype(logits, at),
        None if bias is None else _plane(bias, (E,), "float32", at, "bias"), _plane(ids, (T, k), "int32", at, "ids"),
        _plane(dweights, (T, k), "float32", at, "dweights"), dlogits.data_ptr(),
        _rows(dlogits, T, E, at, "dlogits"), T, E, k, _score(score, at), 1 if renorm else 0, scale,
        _on(logits, stream)), at)
    return dlogits


def moe_experts(gate, up, down, x, ids, weights, offsets, slots, out, stream=None):
    """out [T, D] = the routed experts' gated products of x [T, D] (see include/tq2.h); ids, weights, offsets and
    slots as :func:`moe_route` wrote them."""
    T, D = x.shape
    k = ids.shape[1]
    at = "moe_experts"
    if out.dtype is not x.dtype:
        raise TypeError("moe_experts: x and out must have the same dtype")
    _check((_lib or load()).moe_experts(
        gate.handle, up.handle, down.handle, x.data_ptr(), _rows(x, T, gate.K, at, "x"), _dtype(x, at),
        _plane(ids, (T, k), "int32", at, "ids"), _plane(weights, (T, k), "float32", at, "weights"),
        _plane(offsets, (gate.E + 1,), "int32", at, "offsets"), _plane(slots, (T * k,), "int32", at, "slots"),
        out.data_ptr(), _rows(out, T, D, at, "out"), T, k, _on(x, stream)), at)
    return out


class KV8Cache:
    """A pool of blocks of 8-bit keys and values in the caller's memory (kept alive): ``codes`` uint8
    [blocks, 2, heads, tokens, dim], ``scales`` float32 [blocks, 2, heads], marshalled once."""

    def __init__(self, codes, scales):
        if codes.dim() != 5 or codes.shape[1] != 2:
            raise ValueError(f"KV8Cache: codes must be [blocks, 2, heads, tokens, dim], got {list(codes.shape)}")
        self.blocks, _, self.heads, self.tokens, self.dim = codes.shape
        self.codes, self.scales = codes, scales
        self._c = _Kv8Cache(_plane(codes, tuple(codes.shape), "uint8", "KV8Cache", "codes"),
                            _plane(scales, tuple(codes.shape)[:3], "float32", "KV8Cache", "scales"),
                            self.blocks, self.heads, self.tokens, self.dim)
        self._at = ctypes.addressof(self._c)


class KV8Batch:
    """The sequences of a call in the caller's memory (kept alive; what it holds may change between
    calls): ``table`` int32 [seqs, width] with rows of any stride, ``offsets`` int32 [seqs + 1], ``lens`` int32 [seqs]."""

    def __init__(self, table, offsets, lens):
        if table.dim() != 2:
            raise ValueError(f"KV8Batch: table must be [seqs, width], got {list(table.shape)}")
        self.seqs, self.width = table.shape
        ld = _rows(table, self.seqs, self.width, "KV8Batch", "table")
        self.table, self.offsets, self.lens = table, offsets, lens
        at = _plane(offsets, (self.seqs + 1,), "int32", "KV8Batch", "offsets")
        if table.dtype is not _names["int32"]:
            raise ValueError(f"KV8Batch: table must be int32, got {table.dtype}")
        self._c = _Kv8Batch(table.data_ptr(), ld, at, _plane(lens, (self.seqs,), "int32", "KV8Batch", "lens"),
                            self.width, self.seqs)
        self._at = ctypes.addressof(self._c)


def _heads(t, rows, heads, dim, where, name):
    """Address and strides of a [rows, heads, dim] tensor whose heads' elements are neighbours."""
    if t.shape != (rows, heads, dim):
        raise ValueError(f"{where}: {name} must be [{rows}, {heads}, {dim}], got {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{where}: {name} must be on the GPU")
    st, sh, inner = t.stride()
    if inner != 1:
        raise ValueError(f"{where}: the elements of a head of {name} must be neighbours")
    return t.data_ptr(), st, sh


def _kv8_move(fn, where, cache, batch, k, v, stream):
    if v.dtype is not k.dtype:
        raise TypeError(f"{where}: k and v must have the same dtype")
    T = k.shape[0]
    _check(fn(cache._at, batch._at, *_heads(k, T, cache.heads, cache.dim, where, "k"),
              *_heads(v, T, cache.heads, cache.dim, where, "v"), _dtype(k, where), T, _on(k, stream)), where)
    return k, v


def kv8_write(cache, batch, k, v, stream=None):
    """Quantise the sequences' last tokens ``k``, ``v`` [T, heads, dim] into their blocks (see include/tq2.h)."""
    return _kv8_move((_lib or load()).kv8_write, "kv8_write", cache, batch, k, v, stream)


def kv8_read(cache, batch, k, v, stream=None):
    """The sequences' last tokens as values, into ``k`` and ``v`` [T, heads, dim]."""
    return _kv8_move((_lib or load()).kv8_read, "kv8_read", cache, batch, k, v, stream)


def kv8_attention(cache, batch, q, out, lse=None, scale=None, causal=True, window=0, max_q=None, stream=None):
    """Attention of the sequences' last tokens ``q`` [T, Hq, dim] over the cache into ``out`` [T, Hq, dim] and,
    unless None, ``lse`` float32 [T, Hq] (see include/tq2.h).  scale: dim ** -0.5 if None; max_q: a bound of a
    sequence's rows, 1 when decoding (without one, a batch of more than 32 rows in all counts as a prompt, and is slower)."""
    at = "kv8_attention"
    T, Hq, D = q.shape
    if out.dtype is not q.dtype:
        raise TypeError("kv8_attention: q and out must have the same dtype")
    _check((_lib or load()).kv8_attention(
        cache._at, batch._at, *_heads(q, T, Hq, cache.dim, at, "q"), *_heads(out, T, Hq, cache.dim, at, "out"),
        _dtype(q, at), None if lse is None else _plane(lse, (T, Hq), "float32", at, "lse"), T, Hq,
        D ** -0.5 if scale is None else scale, 1 if causal else 0, window, max_q or 0, _on(q, stream)), at)
    return out


def debug_wait_timeout(limit_ns, stream=None):
    """Launch the test kernel whose bounded wait runs out after ``limit_ns``
    (see include/tq2.h); the next :func:`device_status` raises TQ2_ETIMEOUT."""
    _check(load().tq2_debug_wait_timeout(int(limit_ns), _stream(stream)), "tq2_debug_wait_timeout")


def device_status(stream=None):
    """Synchronize and raise if a kernel recorded a bounded-wait timeout."""
    _check(load().tq2_device_status(_stream(stream)), "tq2_device_status")


def release_scratch():
    """Give back the device memory that the library keeps for the scratch of later calls."""
    _check(load().tq2_release_scratch(), "tq2_release_scratch")
