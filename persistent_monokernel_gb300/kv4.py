"""A KV cache of one layer held in 4 bits (lf_kv4_append / _read / _attend of include/lf.h).

Rows of K and V are stored as E2M1 codes with one E4M3 scale per 16 values, 4.5
bits per value.  The class owns the four byte tensors and marshals arguments;
quantising, reading back and the attention run in the CUDA library, on the
current stream of the cache's device or the one passed.
"""
from __future__ import annotations

import ctypes as C


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
_DTYPES = {}        # torch dtype -> code, filled at first use (the package imports without torch)


def _dtype_code(dt):
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})
    code = _DTYPES.get(dt)
    if code is None:
        raise ValueError(f"dtype {dt}: float16, bfloat16 or float32 is needed")
    return code


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
        import torch
        if k_codes.dim() != 3:
            raise ValueError("codes are [n_kv_heads, max_seq, head_dim / 2]")
        h, s, half = k_codes.shape
        for t, width in ((k_codes, half), (k_scales, half // 8), (v_codes, half), (v_scales, half // 8)):
            if not (t.is_cuda and t.dtype == torch.uint8 and t.is_contiguous() and t.device == k_codes.device
                    and tuple(t.shape) == (h, s, width)):
                raise ValueError("codes [n_kv_heads, max_seq, head_dim / 2] and scales [n_kv_heads, max_seq, "
                                 "head_dim / 16] must be contiguous CUDA torch.uint8 tensors on one device")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.n_kv_heads, self.max_seq, self.head_dim = h, s, 2 * half
        self.device = k_codes.device
        self._c = lf_kv4(h, 2 * half, s, k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                         v_scales.data_ptr())
        self._ref = C.byref(self._c)

    @property
    def nbytes(self) -> int:
        return sum(t.numel() for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales))

    def _rows(self, t, heads, n, what) -> lf_rows:
        shape = t.shape
        if len(shape) != 3 or shape[2] != self.head_dim or (heads is not None and shape[1] != heads) or \
                (n is not None and shape[0] != n):
            raise ValueError(f"{what} is {tuple(shape)}: [n, heads, {self.head_dim}] is needed")
        if t.device != self.device:
            raise ValueError(f"{what} is on {t.device}, the cache on {self.device}")
        ts, hs, es = t.stride()
        if es != 1:
            raise ValueError(f"{what}'s last dimension must be contiguous")
        # the stride of a dimension of one is never used (and may be anything)
        return lf_rows(t.data_ptr(), _dtype_code(t.dtype), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0)

    def _run(self, call, stream):
        """call(stream pointer) with the cache's device current; allocations inside belong to the stream."""
        import torch
        if stream is None:
            if torch.cuda.current_device() == self.device.index:
                return call(torch.cuda.current_stream().cuda_stream)
            with torch.cuda.device(self.device):
                return call(torch.cuda.current_stream().cuda_stream)
        if stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {self.device}")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)

    def append(self, k, v, pos: int, stream=None) -> None:
        """Quantise k, v [n, n_kv_heads, head_dim] into positions pos .. pos + n - 1."""
        n = k.shape[0]
        kr, vr = self._rows(k, self.n_kv_heads, None, "k"), self._rows(v, self.n_kv_heads, n, "v")

        def call(sp):
            _check(_lib().lf_kv4_append(self._ref, C.byref(kr), C.byref(vr), n, int(pos), sp), "lf_kv4_append")
        self._run(call, stream)

    def read(self, pos: int, n: int, dtype=None, out=None, stream=None):
        """(k, v) [n, n_kv_heads, head_dim]: the values of positions pos .. pos + n - 1 (float16 unless `dtype`
        says otherwise; `out` is a pair of tensors to write to)."""
        import torch

        def call(sp):
            pair = out
            if pair is None:
                pair = tuple(torch.empty(max(0, int(n)), self.n_kv_heads, self.head_dim, dtype=dtype or torch.float16,
                                         device=self.device) for _ in range(2))
            kr, vr = (self._rows(t, self.n_kv_heads, max(0, int(n)), w) for t, w in zip(pair, ("k", "v")))
            _check(_lib().lf_kv4_read(self._ref, C.byref(kr), C.byref(vr), int(n), int(pos), sp), "lf_kv4_read")
            return pair
        return self._run(call, stream)

    def attend(self, q, pos: int, length: int | None = None, window: int = 0, scale: float = 0.0, out=None,
               stream=None):
        """Causal attention of q [n, n_heads, head_dim], whose rows stand at positions pos .. pos + n - 1, over the
        cached positions 0 .. length - 1 (pos + n unless given); window W > 0 leaves each row the W most recent.
        A row that sees nothing gives zeros.  Returns [n, n_heads, head_dim] in q's dtype."""
        import torch
        n, pos = q.shape[0], int(pos)
        qr = self._rows(q, None, None, "q")

        def call(sp):
            o = torch.empty(q.shape, dtype=q.dtype, device=self.device) if out is None else out
            orow = self._rows(o, q.shape[1], n, "out")
            args = lf_kv4_query(qr, orow, q.shape[1], n, pos, pos + n if length is None else int(length), int(window),
                                float(scale))
            ref, need, lib = C.byref(args), C.c_int64(), _lib()
            _check(lib.lf_kv4_workspace(self._ref, ref, C.byref(need)), "lf_kv4_attend")
            # scratch of this call alone: no two streams or captured graphs share it
            ws = torch.empty(need.value, dtype=torch.uint8, device=self.device) if need.value else None
            _check(lib.lf_kv4_attend(self._ref, ref, ws.data_ptr() if need.value else None, need.value, sp),
                   "lf_kv4_attend")
            return o
        return self._run(call, stream)


def _check(status: int, where: str) -> None:
    if status:
        from . import LFError
        raise LFError(status, where)


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        from . import lib
        _loaded = lib()
    return _loaded
