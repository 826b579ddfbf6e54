"""The paged KV cache's operators from their definitions, in lists and 64 bits, and how far off the kernels may be."""
import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def cdiv(a, b):
    return -(-a // b)


class Batch:
    """Page tables in lists: what a plan does, one page at a time."""

    def __init__(self, n_seqs, max_pages, n_pages, page):
        self.tables = [[0] * max_pages for _ in range(n_seqs)]
        self.lens, self.free, self.page, self.max_pages = [0] * n_seqs, list(range(n_pages - 1, -1, -1)), page, max_pages

    def plan(self, n_new, max_tokens, keep=None):
        """(slots, positions, offsets, failed)"""
        n, P = len(self.lens), self.page
        keep = self.lens if keep is None else keep
        kept = [min(a, b) for a, b in zip(self.lens, keep)]
        after = [a + b for a, b in zip(kept, n_new)]
        given = [self.tables[i][j] for i in range(n) for j in range(cdiv(kept[i], P), cdiv(self.lens[i], P))]
        need = sum(cdiv(a, P) - cdiv(k, P) for a, k in zip(after, kept))
        if need > len(self.free) + len(given) or sum(n_new) > max_tokens or max(after, default=0) > self.max_pages * P:
            return [-1] * max_tokens, [0] * max_tokens, [0] * (n + 1), True
        self.free += reversed(given)
        slots, positions, offsets = [], [], [0]
        for i in range(n):
            for p in range(kept[i], after[i]):
                if p % P == 0:
                    self.tables[i][p // P] = self.free.pop()
                slots.append(self.tables[i][p // P] * P + p % P)
                positions.append(p)
            self.lens[i] = after[i]
            offsets.append(len(slots))
        rest = max_tokens - len(slots)
        return slots + [-1] * rest, positions + [0] * rest, offsets, False


def visible(tables, lens, i, page, window, n_pages):
    """(pages, places) of the positions that row i sees."""
    n = int(lens[i])
    lo = max(0, n - window) if window else 0
    hi = min(n, tables.shape[1] * page)
    j = torch.arange(lo, max(lo, hi), device=tables.device)
    ids = tables[i].long()[j // page] if len(j) else j
    fine = (ids >= 0) & (ids < n_pages)
    return ids[fine], (j % page)[fine]


def attend(q, k, v, tables, lens, window=0, scale=0.0):
    """(outputs, bounds of their error) [n, heads, head_dim] in 64 bits; k, v [n_pages, n_kv_heads, page, head_dim].

    With weights p_j and y = sum p_j v_j, weights that are off by a factor 1 + d_j move y by at most max|d| M,
    M = sum p_j |v_j - y|, where they are divided by their own sum, and 2 max|d| M covers a sum of others.  d holds
      - the score's error: head_dim products summed in 32 bits with cut sums, 2^-23 of sum |q_d k_d| a step; q as the sum
        of two FP16 terms (2^-22, and 2^-25 of the row's largest value where a term runs out of exponents) or three
        BF16 ones (2^-24); the exponent's arithmetic, 2^-22 of the score and its largest; exp2 itself, 2^-21;
      - the rounding of P: two FP16 terms 2^-22, two BF16 terms 2^-16 (three with FP32 queries, 2^-24).
    FP16 terms of P end at 2^-24, half a step 2^-25 of a largest P of 2^6 at least: n 2^-31 max|v|.  O's own sum:
    n / 8 steps of 2^-23 of sum p_j |v_j| (and 64 for the joins); then the output's half step."""
    n_pages, hkv, page, hd = k.shape
    n, heads, _ = q.shape
    group, f32 = heads // hkv, q.dtype == torch.float32
    scale = scale or 1 / math.sqrt(hd)
    out = torch.zeros(n, heads, hd, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    p_step = 2.0 ** -22 if f32 or k.dtype == torch.float16 else 2.0 ** -16
    for i in range(n):
        pages, places = visible(tables, lens, i, page, window, n_pages)
        if not len(pages):
            continue
        m = len(pages)
        for h in range(hkv):
            kk, vv = k[pages, h, places].double(), v[pages, h, places].double()
            qq = q[i, h * group:(h + 1) * group].double()
            s = qq @ kk.T * scale
            p = torch.softmax(s, -1)
            y = p @ vv
            spread = torch.stack([p[g] @ (vv - y[g]).abs() for g in range(group)])
            d = abs(scale) * (qq.abs() @ kk.abs().T) * (hd * 2.0 ** -23 + (2.0 ** -22 if f32 else 0))
            if f32:
                d += abs(scale) * 2.0 ** -25 * qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)
            d = (d + 2.0 ** -22 * (s.abs() + s.abs().amax(-1, keepdim=True))).amax(-1, keepdim=True) + 2.0 ** -21
            b = 2 * d * spread + p_step * (1 + d) * spread
            if k.dtype == torch.float16:
                b = b + m * 2.0 ** -31 * vv.abs().amax()
            b = b + (m / 8 + 64) * 2.0 ** -23 * (p @ vv.abs())
            rows = slice(h * group, (h + 1) * group)
            out[i, rows] = y
            bound[i, rows] = b + HALF_STEP[q.dtype] * (y.abs() + b) + (2.0 ** -25 if q.dtype == torch.float16 else 0)
    return out, bound


def pools(n_pages, hkv, page, hd, dtype, seed, by_head=True, fill=float("nan")):
    """K and V pools, all `fill`, in either order of heads and positions."""
    g = torch.Generator("cuda").manual_seed(seed)
    out = []
    for _ in range(2):
        shape = (n_pages, hkv, page, hd) if by_head else (n_pages, page, hkv, hd)
        t = torch.full(shape, fill, dtype=dtype, device="cuda")
        out.append(t if by_head else t.transpose(1, 2))
    return *out, g


def case(lens, heads, hkv, hd, page, dtype, q_dtype, seed=0, by_head=True, width=None, spread=1.0):
    """A cache whose pools hold NaN wherever no row's positions lie, its tables (entries behind a row's pages are no
    pages at all), lengths and queries."""
    width = max(cdiv(max(max(lens), 1), page) if width is None else width, 1)
    counts = [cdiv(n, page) for n in lens]
    n_pages = sum(counts) + 2
    k, v, g = pools(n_pages, hkv, page, hd, dtype, seed, by_head)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    tables = torch.full((len(lens), max(width, max(counts, default=0))), -7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(lens):
        for j in range(counts[i]):
            tables[i, j] = order[at]
            rows = min(page, n - j * page)
            for t in (k, v):
                t[order[at], :, :rows] = (spread * torch.randn(hkv, rows, hd, generator=g, device="cuda")).to(dtype)
            at += 1
    q = torch.randn(len(lens), heads, hd, generator=g, device="cuda").to(q_dtype)
    return q, k, v, tables[:, :width].cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def check(got, want, bound):
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all())
    worst = (err - bound).max().item()
    assert worst <= 0, (worst, err.max().item(), (err / bound.clamp(min=1e-300)).max().item())
