"""A KV cache of one layer held in 4 bits (lf_kv4_append / _read / _attend of include/lf.h).

Rows of K and V are stored as E2M1 codes with one E4M3 scale per 16 values, 4.5
bits per value.  The class owns the four byte tensors and marshals arguments;
quantising, reading back and the attention run in the CUDA library, on the
current stream of the cache's device or the one passed.
"""
from __future__ import annotations

import ctypes as C
import struct


class lf_kv4(C.Structure):
    _fields_ = [("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("max_seq", C.c_int32),
                ("k_codes", C.c_void_p), ("k_scales", C.c_void_p), ("v_codes", C.c_void_p), ("v_scales", C.c_void_p)]


class lf_rows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("dtype", C.c_int32), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class lf_kv4_query(C.Structure):
    _fields_ = [("q", lf_rows), ("out", lf_rows), ("n_heads", C.c_int32), ("n", C.c_int32), ("pos", C.c_int32),
                ("length", C.c_int32), ("window", C.c_int32), ("scale", C.c_float)]


F16, BF16, F32 = 0, 1, 2
BLOCK = 16          # values that share a scale
_INT = 2 ** 31
_byref = C.byref
_torch = _lib = _append = _read = _attend = _codes = _raw_stream = _current_device = None
# The argument structures as bytes, packed in one call (a ctypes structure takes a microsecond to fill, and a decode
# step's kernels take a few on the GPU): data, dtype, token_stride, head_stride; then the query's other fields.
_ROWS = struct.Struct("@Piqq")
_QUERY = struct.Struct("@PiqqPiqqiiiiif")


def _load():
    """torch and the library, once, at the first cache (the package imports without torch)."""
    global _torch, _lib, _append, _read, _attend, _codes, _raw_stream, _current_device
    import torch

    from . import lib
    _lib = lib()
    assert _ROWS.size == C.sizeof(lf_rows) and _QUERY.size == C.sizeof(lf_kv4_query)
    # prototypes of their own that take the packed bytes
    calls = [_lib["lf_kv4_append"], _lib["lf_kv4_read"], _lib["lf_kv4_attend"]]
    for f in calls[:2]:
        f.argtypes = [C.c_void_p, C.c_char_p, C.c_char_p, C.c_int32, C.c_int32, C.c_void_p]
    calls[2].argtypes = [C.c_void_p, C.c_char_p, C.c_void_p, C.c_int64, C.c_void_p]
    for f in calls:
        f.restype = C.c_int
    _append, _read, _attend = calls
    _codes = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
    # the plain functions behind torch.cuda.current_stream and current_device (a Stream object costs three microseconds)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda i: torch.cuda.current_stream(i).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch


class KV4Cache:
    """K and V of one layer for positions 0 .. max_seq - 1, `n_kv_heads` heads of `head_dim` (64 or 128) values.

    Tensors passed to the calls are CUDA tensors [n, heads, head_dim] on the cache's device with a contiguous last
    dimension, 16-byte aligned rows and any other strides (a slice of a fused projection, or a transposed
    [heads, n, head_dim] tensor); what the library refuses raises LFError.
    """

    def __init__(self, n_kv_heads: int, head_dim: int, max_seq: int, device="cuda"):
        import torch
        parts = [torch.zeros(int(n_kv_heads), int(max_seq), int(head_dim) // w, dtype=torch.uint8, device=device)
                 for w in (2, BLOCK, 2, BLOCK)]
        self._set(*parts)

    @classmethod
    def wrap(cls, k_codes, k_scales, v_codes, v_scales) -> "KV4Cache":
        """A cache over four existing uint8 tensors: codes [n_kv_heads, max_seq, head_dim / 2] and scales
        [n_kv_heads, max_seq, head_dim / 16], contiguous, on one CUDA device."""
        self = cls.__new__(cls)
        self._set(k_codes, k_scales, v_codes, v_scales)
        return self

    def _set(self, k_codes, k_scales, v_codes, v_scales) -> None:
        if _torch is None:
            _load()
        if k_codes.dim() != 3:
            raise ValueError("codes are [n_kv_heads, max_seq, head_dim / 2]")
        h, s, half = k_codes.shape
        if max(h, s) >= _INT:
            raise ValueError(f"{h} heads, {s} positions: 32 bits are needed")
        for t, width in ((k_codes, half), (k_scales, half // 8), (v_codes, half), (v_scales, half // 8)):
            if not (t.is_cuda and t.dtype == _torch.uint8 and t.is_contiguous() and t.device == k_codes.device
                    and tuple(t.shape) == (h, s, width)):
                raise ValueError("codes [n_kv_heads, max_seq, head_dim / 2] and scales [n_kv_heads, max_seq, "
                                 "head_dim / 16] must be contiguous CUDA torch.uint8 tensors on one device")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.n_kv_heads, self.max_seq, self.head_dim = h, s, 2 * half
        self.device = k_codes.device
        self._index = k_codes.get_device()
        self._c = lf_kv4(h, 2 * half, s, k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                         v_scales.data_ptr())
        self._ref, self._addr = _byref(self._c), C.addressof(self._c)
        self._scratch = None, 0     # shape of the last query that needed scratch, and how much

    @property
    def nbytes(self) -> int:
        return sum(t.numel() for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales))

    def _rows(self, t, n, heads, what):
        """The fields of lf_rows for t [n, heads, head_dim]."""
        stride = t.stride()
        code = _codes.get(t.dtype)
        if t.shape != (n, heads, self.head_dim) or t.get_device() != self._index or stride[2] != 1 or code is None:
            raise ValueError(f"{what} is {t.dtype} {tuple(t.shape)}, strides {stride}, on {t.device}: [{n}, {heads}, "
                             f"{self.head_dim}] float16, bfloat16 or float32 with a contiguous last dimension on "
                             f"{self.device} is needed")
        # the stride of a dimension of one is never used (and may be anything)
        return t.data_ptr(), code, stride[0] if n > 1 else 0, stride[1] if heads > 1 else 0

    def _elsewhere(self, call, stream, args):
        """The call again with the cache's device, and the stream if one is passed, current: what it allocates belongs
        to that stream."""
        if stream is None:
            with _torch.cuda.device(self.device):
                return call(*args)
        if stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {self.device}")
        with _torch.cuda.stream(stream):
            return call(*args)

    def append(self, k, v, pos: int, stream=None) -> None:
        """Quantise k, v [n, n_kv_heads, head_dim] into positions pos .. pos + n - 1."""
        if stream is not None or _current_device() != self._index:
            return self._elsewhere(self.append, stream, (k, v, pos))
        n, h = len(k), self.n_kv_heads
        if not (-_INT < pos < _INT and n < _INT):
            raise ValueError(f"pos {pos}, {n} rows: 32 bits are needed")
        status = _append(self._addr, _ROWS.pack(*self._rows(k, n, h, "k")), _ROWS.pack(*self._rows(v, n, h, "v")), n, pos,
                         _raw_stream(self._index))
        if status:
            _fail(status, "lf_kv4_append")

    def read(self, pos: int, n: int, dtype=None, out=None, stream=None):
        """(k, v) [n, n_kv_heads, head_dim]: the values of positions pos .. pos + n - 1 (float16 unless `dtype`
        says otherwise; `out` is a pair of tensors to write to)."""
        if stream is not None or _current_device() != self._index:
            return self._elsewhere(self.read, stream, (pos, n, dtype, out))
        h = self.n_kv_heads
        if not (-_INT < pos < _INT and -_INT < n < _INT):
            raise ValueError(f"pos {pos}, n {n}: 32 bits are needed")
        if out is None:
            shape, dtype = (max(n, 0), h, self.head_dim), dtype or _torch.float16
            k = _torch.empty(shape, dtype=dtype, device=self.device)
            v = _torch.empty(shape, dtype=dtype, device=self.device)
        else:
            k, v = out
        status = _read(self._addr, _ROWS.pack(*self._rows(k, max(n, 0), h, "k")),
                       _ROWS.pack(*self._rows(v, max(n, 0), h, "v")), n, pos, _raw_stream(self._index))
        if status:
            _fail(status, "lf_kv4_read")
        return k, v

    def attend(self, q, pos: int, length: int | None = None, window: int = 0, scale: float = 0.0, out=None,
               stream=None):
        """Causal attention of q [n, n_heads, head_dim], whose rows stand at positions pos .. pos + n - 1, over the
        cached positions 0 .. length - 1 (pos + n unless given); window W > 0 leaves each row the W most recent.
        A row that sees nothing gives zeros.  Returns [n, n_heads, head_dim] in q's dtype."""
        if stream is not None or _current_device() != self._index:
            return self._elsewhere(self.attend, stream, (q, pos, length, window, scale, out))
        n, heads, _ = shape = q.shape
        rows = self._rows(q, n, heads, "q")
        if out is None:
            out = _torch.empty(shape, dtype=q.dtype, device=self.device)
        try:
            args = _QUERY.pack(*rows, *self._rows(out, n, heads, "out"), heads, n, pos, pos + n if length is None else length,
                               window, scale)
        except struct.error as err:
            raise ValueError(f"pos {pos}, length {length}, window {window}, scale {scale}: {err}") from None
        # Scratch (long contexts and large blocks need some) belongs to this call alone: no two streams or captured
        # graphs share it.  Its size is asked for when a call like the last one turns out not to have enough.
        key, size = self._scratch
        if key != (n, heads):
            size = 0
        # (Held until the launch: another thread on this stream may be given what is let go before it.)
        ws = _torch.empty((size,), dtype=_torch.uint8, device=self.device) if size else None
        status = _attend(self._addr, args, ws.data_ptr() if size else None, size, _raw_stream(self._index))
        if status:
            status = self._attend_with_workspace(args, status, (n, heads))
            if status:
                _fail(status, "lf_kv4_attend")
        return out

    def _attend_with_workspace(self, args, status, key):
        """The call again with the scratch it needs, if that is what it lacked."""
        query, need = lf_kv4_query.from_buffer_copy(args), C.c_int64()
        if _lib.lf_kv4_workspace(self._ref, _byref(query), _byref(need)) or not need.value:
            return status
        self._scratch = key, need.value
        ws = _torch.empty((need.value,), dtype=_torch.uint8, device=self.device)
        return _attend(self._addr, args, ws.data_ptr(), need.value, _raw_stream(self._index))

    def sync(self) -> int:
        """Synchronise the current stream of the cache's device: 0, or LF_ERR_TIMEOUT (6) if a device-side wait of an
        attend call ran out since the last sync (lf_kv4_status)."""
        with _torch.cuda.device(self.device):
            return int(_lib.lf_kv4_status(_raw_stream(self._index)))


def _fail(status: int, where: str) -> None:
    from . import LFError
    raise LFError(status, where)
