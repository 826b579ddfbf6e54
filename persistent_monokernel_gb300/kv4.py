"""A KV cache of one layer held in 4 bits (lf_kv4_append / _read / _attend of include/lf.h).

Rows of K and V are stored as E2M1 codes with one E4M3 scale per 16 values, 4.5
bits per value.  The class holds the four byte tensors; _lft.so marshals its
calls, and quantising, reading back and the attention run in the CUDA library,
on the current stream of the cache's device or the one passed.
"""
from __future__ import annotations

import ctypes as C
import re
import sys
import threading


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
_BUILD = "build it with `python -m persistent_monokernel_gb300.build`"
_TIMEOUT = 6        # LF_ERR_TIMEOUT
_torch = _lib = _calls = _codes = None
_told, _told_lock = {}, threading.Lock()   # device: how often lf_kv4_status has told of a wait that ran out


def _load():
    """torch, the library and the module of its calls, once, at the first cache (the package imports without torch)."""
    global _torch, _lib, _calls, _codes
    import torch

    from . import lib
    _lib = lib()
    try:
        from . import _lft
    except ImportError as e:
        raise ImportError(f"_lft.so cannot be loaded ({e}): {_BUILD}") from e
    have = (".".join(re.findall(r"\d+", torch.__version__)[:3]), sys.hexversion >> 16)
    if _lft.made_for != have:
        raise ImportError(f"_lft.so was built for torch {_lft.made_for[0]} and Python {_lft.made_for[1]:#x}, not for "
                          f"{have[0]} and {have[1]:#x}: {_BUILD}")
    _lft.bind(*(C.cast(getattr(_lib, "lf_kv4_" + f), C.c_void_p).value for f in ("append", "read", "attend", "workspace")),
              _fail)
    _calls = _lft
    _codes = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
    _torch = torch


class KV4Cache:
    """K and V of one layer for positions 0 .. max_seq - 1, `n_kv_heads` heads of `head_dim` (64 or 128) values.

    Tensors passed to the calls are CUDA tensors [n, heads, head_dim] on the cache's device with a contiguous last
    dimension, 16-byte aligned rows and any other strides (a slice of a fused projection, or a transposed
    [heads, n, head_dim] tensor); what the library refuses raises LFError.  The calls form no gradients: where autograd
    is on, a tensor that requires one raises ValueError.

    A call with stream=s queues its work on s and returns.  Its tensors and the cache may be let go of at once (on an
    ExternalStream, whose life torch does not know, once the work is done); what it returns belongs to s, as with any
    torch operation under torch.cuda.stream(s).
    """

    def __init__(self, n_kv_heads: int, head_dim: int, max_seq: int, device="cuda"):
        import torch
        parts = [torch.zeros(int(n_kv_heads), int(max_seq), int(head_dim) // w, dtype=torch.uint8, device=device)
                 for w in (2, BLOCK, 2, BLOCK)]
        self._set(*parts)

    @classmethod
    def wrap(cls, k_codes, k_scales, v_codes, v_scales) -> "KV4Cache":
        """A cache over four existing uint8 tensors: codes [n_kv_heads, max_seq, head_dim / 2] and scales
        [n_kv_heads, max_seq, head_dim / 16], contiguous, on one CUDA device.  They stay the cache's own: another
        four are another cache."""
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
        self._parts = (k_codes, k_scales, v_codes, v_scales)
        self.n_kv_heads, self.max_seq, self.head_dim = h, s, 2 * half
        self.device = k_codes.device
        self._heard = _told.get(self.device, 0)
        self._handle = _calls.cache(h, 2 * half, s, k_codes.get_device(), *self._parts)

    # the tensors are read where they lie at each call; others cannot take their place
    k_codes, k_scales, v_codes, v_scales = (property(lambda self, i=i: self._parts[i]) for i in range(4))

    @property
    def nbytes(self) -> int:
        return sum(t.numel() for t in self._parts)

    def _elsewhere(self, call, stream, args):
        """The call again with the cache's device, and the stream if one is passed, current: what it allocates belongs
        to that stream.  What the call reads and writes is marked as in use there, so that memory that the caller lets
        go of before the stream is done is not given to another."""
        if stream is None:
            with _torch.cuda.device(self.device):
                return call(*args)
        if stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {self.device}")
        with _torch.cuda.stream(stream):
            got = call(*args)
        if not isinstance(stream, _torch.cuda.ExternalStream):   # (which may be gone when the memory is let go of)
            for t in (*self._parts, *_tensors(args)):
                t.record_stream(stream)
        return got

    def append(self, k, v, pos: int, stream=None) -> None:
        """Quantise k, v [n, n_kv_heads, head_dim] into positions pos .. pos + n - 1."""
        if stream is not None or _calls.append(self._handle, k, v, pos) is NotImplemented:
            self._elsewhere(self.append, stream, (k, v, pos))

    def read(self, pos: int, n: int, dtype=None, out=None, stream=None):
        """(k, v) [n, n_kv_heads, head_dim]: the values of positions pos .. pos + n - 1 (float16 unless `dtype`
        says otherwise; `out` is a pair of tensors to write to)."""
        code = F16 if dtype is None else _codes.get(dtype)
        if code is None:
            raise ValueError(f"{dtype}: float16, bfloat16 or float32 is needed")
        k, v = (None, None) if out is None else out
        if stream is None and (got := _calls.read(self._handle, pos, n, code, k, v)) is not NotImplemented:
            return got
        return self._elsewhere(self.read, stream, (pos, n, dtype, out))

    def attend(self, q, pos: int, length: int | None = None, window: int = 0, scale: float = 0.0, out=None,
               stream=None):
        """Causal attention of q [n, n_heads, head_dim], whose rows stand at positions pos .. pos + n - 1, over the
        cached positions 0 .. length - 1 (pos + n unless given); window W > 0 leaves each row the W most recent; scale
        0 selects 1 / sqrt(head_dim).  A row that sees nothing gives zeros.  Returns [n, n_heads, head_dim] in q's dtype:
        a new tensor, or `out`, which must not overlap q."""
        if stream is None:
            got = _calls.attend(self._handle, q, pos, length, window, scale, out)
            if got is not NotImplemented:
                return got
        return self._elsewhere(self.attend, stream, (q, pos, length, window, scale, out))

    def sync(self) -> int:
        """Synchronise the current stream of the cache's device: 0, or LF_ERR_TIMEOUT (6) if a device-side wait of an
        attend call on that device, of this cache or another, ran out since this cache's last sync (lf_kv4_status,
        which tells once: every cache of the process is told)."""
        with _torch.cuda.device(self.device):
            status = int(_lib.lf_kv4_status(_torch.cuda.current_stream().cuda_stream))
        with _told_lock:
            told = _told.get(self.device, 0)
            if status == _TIMEOUT:
                told = _told[self.device] = told + 1
            elif status == 0 and told != self._heard:
                status = _TIMEOUT
            self._heard = told
        return status


def _tensors(args):
    """The tensors among a call's arguments, those of a pair (read's out) too."""
    for a in args:
        if isinstance(a, _torch.Tensor):
            yield a
        elif isinstance(a, (tuple, list)):
            yield from _tensors(a)


def _fail(status: int, where: str) -> None:
    from . import LFError
    raise LFError(status, where)
