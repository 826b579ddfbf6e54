"""A KV cache that many sequences share, in pages (lf_paged_plan / _append / _attend of include/lf.h).

PageTables holds which pages each sequence of a batch owns and plans a step on
the GPU; PagedKVCache holds the K and V of one layer.  The classes hold tensors;
_lft.so marshals their calls, and the work runs in the CUDA library, on the
current stream of the tensors' device or the one passed.  A decode step, with
nothing on the host:

    slots, positions, offsets = tables.plan(n_new, max_tokens)     # once, for all layers
    cache.append(k, v, slots)                                      # per layer
    out = cache.attend(q, tables.tables[:, :pages], tables.lens)

`pages` is a bound of what any row needs that the host knows (all columns are one, too): the lengths are the device's,
and the attention's launch goes by the table's width.
"""
from __future__ import annotations

import ctypes as C

from . import kv4
from .kv4 import OnStream, lf_rows


class lf_paged(C.Structure):
    _fields_ = [("n_pages", C.c_int32), ("n_kv_heads", C.c_int32), ("page", C.c_int32), ("head_dim", C.c_int32),
                ("dtype", C.c_int32), ("k", C.c_void_p), ("v", C.c_void_p), ("page_stride", C.c_int64),
                ("head_stride", C.c_int64), ("pos_stride", C.c_int64)]


class lf_page_tables(C.Structure):
    _fields_ = [("n_seqs", C.c_int32), ("max_pages", C.c_int32), ("n_pages", C.c_int32), ("page", C.c_int32),
                ("tables", C.c_void_p), ("table_stride", C.c_int64), ("lens", C.c_void_p), ("free_pages", C.c_void_p),
                ("n_free", C.c_void_p), ("status", C.c_void_p)]


class lf_paged_query(C.Structure):
    _fields_ = [("q", lf_rows), ("out", lf_rows), ("n_seqs", C.c_int32), ("n_heads", C.c_int32), ("tables", C.c_void_p),
                ("table_stride", C.c_int64), ("table_width", C.c_int32), ("lens", C.c_void_p), ("window", C.c_int32),
                ("scale", C.c_float)]


class PageTables(OnStream):
    """Which pages of a pool of `n_pages` (of `page` positions, a multiple of 16) each of `n_seqs` sequences owns, at most
    `max_pages` each: int32 CUDA tensors tables [n_seqs, max_pages], lens [n_seqs], and free [n_pages], whose first
    n_free [1] entries are the pages that nobody owns.  All start empty.  One object serves every layer whose pools
    have n_pages pages.

    Calls take a stream as KV4Cache's do.
    """
    _what = "page tables"

    def __init__(self, n_seqs: int, max_pages: int, n_pages: int, page: int = 64, device="cuda"):
        import torch
        tables = torch.zeros(int(n_seqs), int(max_pages), dtype=torch.int32, device=device)
        self._set(tables, torch.zeros(int(n_seqs), dtype=torch.int32, device=device),
                  torch.arange(int(n_pages) - 1, -1, -1, dtype=torch.int32, device=device),
                  torch.full((1,), int(n_pages), dtype=torch.int32, device=device), page)

    @classmethod
    def wrap(cls, tables, lens, free, n_free, page: int) -> "PageTables":
        """Page tables over existing tensors, which stay the object's own."""
        self = cls.__new__(cls)
        self._set(tables, lens, free, n_free, page)
        return self

    def _set(self, tables, lens, free, n_free, page) -> None:
        if kv4._torch is None:
            kv4._load()
        torch = kv4._torch
        page = int(page)
        if not (16 <= page < 2 ** 31 and page % 16 == 0):
            raise ValueError(f"{page} positions per page: a multiple of 16 is needed")
        status = torch.zeros(1, dtype=torch.int32, device=tables.device)
        self._parts = (tables, lens, free, n_free, status)
        self._handle = kv4._calls.page_tables(page, *self._parts)
        (self.n_seqs, self.max_pages), self.n_pages = tables.shape, len(free)
        self.page, self.device = page, tables.device

    # the tensors are read where they lie at each call; others cannot take their place
    tables, lens, free, n_free, status = (property(lambda self, i=i: self._parts[i]) for i in range(5))

    def plan(self, n_new, max_tokens: int, keep=None, stream=None):
        """Plan one step on the GPU: row i keeps min(lens[i], keep[i]) positions (all unless `keep` is given), gives
        the pages behind them back, and gets the pages for n_new[i] more; lens becomes the sum (n_new, keep: int32
        [n_seqs]).  keep[i] = 0 ends sequence i, and with n_new[i] lets another take its row; keep[i] < lens[i] takes
        drafted positions back.

        Returns (slots, positions, offsets), int32 parts of one new allocation: the new positions of all rows, packed in
        row order, slots [max_tokens] for PagedKVCache.append, positions [max_tokens] within their sequences, and where
        each row's begin [n_seqs + 1].  Behind the last one slots are -1 and positions 0.

        All or nothing: where the pages, the rows' max_pages or max_tokens do not suffice, nothing changes, all slots
        are -1 and all offsets 0, and sync() on the same stream tells."""
        if stream is None:
            got = kv4._calls.plan(self._handle, n_new, max_tokens, keep)
            if got is not NotImplemented:
                return got
        return self._elsewhere(self.plan, stream, (n_new, max_tokens, keep))

    def sync(self, stream=None) -> int:
        """Synchronise `stream`, or the current stream of the tables' device: 0, or why a plan since the last sync changed
        nothing, LF_ERR_CAPACITY (3) or LF_ERR_INVALID_ARG (1), the first where there were several.  Plans that are
        still to run on other streams are not waited for."""
        if stream is not None:
            return self._elsewhere(self.sync, stream, ())
        with kv4._torch.cuda.device(self.device):
            status = int(self.status.item())
            if status:
                self.status.zero_()
        return status


def _check_pool(shape, dtype) -> None:
    """Raise LFError for contiguous pools [n_pages, n_kv_heads, page, head_dim] that the library refuses: an append of no
    rows checks them and does nothing else (the addresses are any)."""
    from . import lib
    if kv4._torch is None:
        kv4._load()
    code = kv4._codes.get(dtype)
    if code not in (kv4.F16, kv4.BF16) or max(shape) >= 2 ** 31:
        raise ValueError(f"pools {list(shape)} of {dtype}: sizes of 32 bits, float16 or bfloat16 are needed")
    n_pages, heads, page, hd = shape
    pools = lf_paged(n_pages, heads, page, hd, code, 16, 32, heads * page * hd, page * hd, hd)
    status = lib().lf_paged_append(C.byref(pools), None, None, 0, None, None)
    if status:
        kv4._fail(status, "lf_paged")


class PagedKVCache(OnStream):
    """K and V of one layer in `n_pages` pages of `page` positions (a multiple of 16), `n_kv_heads` heads of `head_dim`
    (64 or 128) values in float16 or bfloat16.

    Rows passed to the calls are CUDA tensors [n, heads, head_dim] on the cache's device, of the cache's dtype or
    float32, with a contiguous last dimension, 16-byte aligned rows and any other strides; what the library refuses
    raises LFError.  The calls form no derivatives and take a stream as KV4Cache's do.
    """

    def __init__(self, n_pages: int, n_kv_heads: int, head_dim: int, page: int = 64, dtype=None, device="cuda"):
        import torch
        shape = int(n_pages), int(n_kv_heads), int(page), int(head_dim)
        dtype = dtype or torch.float16
        _check_pool(shape, dtype)                          # before any memory is asked for
        self._set(*(torch.zeros(shape, dtype=dtype, device=device) for _ in range(2)))

    @classmethod
    def wrap(cls, k, v) -> "PagedKVCache":
        """A cache over two existing tensors [n_pages, n_kv_heads, page, head_dim], alike in strides: contiguous, a
        permuted [n_pages, page, n_kv_heads, head_dim], or slices of one that holds both.  They stay the cache's own."""
        self = cls.__new__(cls)
        self._set(k, v)
        return self

    def _set(self, k, v) -> None:
        if kv4._torch is None:
            kv4._load()
        self._handle = kv4._calls.paged(k, v)
        self._parts = (k, v)
        self.n_pages, self.n_kv_heads, self.page, self.head_dim = k.shape
        self.dtype, self.device = k.dtype, k.device

    k, v = (property(lambda self, i=i: self._parts[i]) for i in range(2))

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self._parts)

    def append(self, k, v, slots, stream=None) -> None:
        """Store row t of k and v [n, n_kv_heads, head_dim] at slot slots[t] (int32 [n], as PageTables.plan gives them);
        slots outside the pool store nothing.  float32 rows are rounded to nearest even."""
        if stream is not None or kv4._calls.paged_append(self._handle, k, v, slots) is NotImplemented:
            self._elsewhere(self.append, stream, (k, v, slots))

    def attend(self, q, tables, lens, window: int = 0, scale: float = 0.0, out=None, stream=None):
        """Attention of one query row per sequence, q [n_seqs, n_heads, head_dim], over its first lens[i] positions, which
        lie in the pages tables[i] (int32 [n_seqs, pages], [n_seqs]); window W > 0 leaves the W most recent; scale 0
        selects 1 / sqrt(head_dim).  A row that sees nothing gives zeros; positions behind the table's columns or on
        pages that the pool does not have are left out.  The launch goes by the table's
        width: pass the columns that a bound of the longest row needs (tables[:, :pages]).  Returns [n_seqs, n_heads,
        head_dim] in q's dtype: a new tensor, or `out`, which must not overlap q."""
        if stream is None:
            got = kv4._calls.paged_attend(self._handle, q, tables, lens, window, scale, out)
            if got is not NotImplemented:
                return got
        return self._elsewhere(self.attend, stream, (q, tables, lens, window, scale, out))
