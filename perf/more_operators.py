"""The operators of a paged KV cache that many requests share: their cases and plain forms.

The K and V of one layer lie in a pool of pages of `page` positions, [n_pages,
n_kv_heads, page, head_dim] (or a permuted view of [n_pages, page, n_kv_heads,
head_dim]).  Row i of a batch owns the pages tables[i][0 ..]; its position p is
slot tables[i][p // page] * page + p % page.  Pages that no row owns are the
first n_free entries of `free`, a stack whose top is free[n_free - 1].

  plan     row i keeps min(lens[i], keep[i]) positions and gives the pages behind
           them back, then gets the pages for n_new[i] more; the slot and position
           of each new token, packed by row, and where each row's begin
  append   row t of k and v is stored at slot slots[t] (below 0: nowhere)
  attend   one query row per request over its lens[i] positions (with a window W,
           the W most recent); a row of length 0 gives zeros
  step     the three as a decode step makes them: plan, append, attend
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# query heads, KV heads, head_dim of this repository's decoders (tiny, small, 2.3B, 8B shape), and three generic groupings
HEADS = [(4, 4, 64), (16, 4, 64), (20, 5, 128), (32, 8, 128), (8, 1, 128), (32, 2, 128), (12, 1, 64)]
PAGES = [16, 32, 48, 64, 128, 256]


def _plan(name, rows, top, new, page, fresh=0):
    """rows of up to `top` positions, each to take up to `new` more; every fresh-th row begins anew."""
    c = {"kind": "plan", "rows": rows, "top": top, "new": new, "page": page, "fresh": fresh}
    return dict(c, name=name) if name else c


def _append(name, heads, n, page, cache, dtype, by_head=True):
    c = {"kind": "append", "hkv": heads[1], "hd": heads[2], "n": n, "page": page, "cache": cache, "dtype": dtype, "by_head": by_head}
    return dict(c, name=name) if name else c


def _attend(name, heads, rows, top, page, cache, dtype, window=0, skew=1, by_head=True, kind="attend"):
    """rows of lengths 0 .. top, spread evenly (skew 1) or most of them short (above)."""
    c = {"kind": kind, "hq": heads[0], "hkv": heads[1], "hd": heads[2], "rows": rows, "top": top, "page": page,
         "cache": cache, "dtype": dtype, "window": window, "skew": skew, "by_head": by_head}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of 64 requests: one new position each, a new page for a few
        _plan("plan-64-decode", 64, 4096, 1, 64),
        # drafted tokens of 500 requests taken back and drawn anew, every fifth row given to a new prompt
        _plan("plan-500-prompts", 500, 2048, 333, 16, 5),
        # the new rows of 64 requests: latency only
        _append("append-64", (32, 8, 128), 64, 64, "f16", "f16"),
        # a batch of prompts from a program with FP32 activations
        _append("append-8191", (20, 5, 128), 8191, 16, "f16", "f32", False),
        # one session of the 2.3B decoder right after its 512-token prompt
        _attend("attend-1x512", (20, 5, 128), 1, 512, 64, "f16", "f16"),
        # a few sessions with the FP32 activations of this repository's decoders
        _attend("attend-7x1000-f32", (20, 5, 128), 7, 1000, 16, "f16", "f32"),
        # narrow heads, a sliding window, positions outside heads
        _attend("attend-33x8000-window", (16, 4, 64), 33, 8000, 32, "bf16", "bf16", 1000, 1, False),
        # one long context of the 8B shape: its bytes are all that counts
        _attend("attend-1x131071", (32, 8, 128), 1, 131071, 256, "f16", "f16"),
        # many short requests and a few long ones, wide groups, FP32 queries on a BF16 cache
        _attend("attend-200-skewed-f32", (32, 2, 128), 200, 20000, 48, "bf16", "f32", 0, 4),
        # a full batch of the 8B shape: the largest
        _attend("attend-64x16384", (32, 8, 128), 64, 16384, 64, "bf16", "bf16"),
        # a decode step of a small batch, from lengths to outputs
        _attend("step-24x3000", (20, 5, 128), 24, 3000, 64, "f16", "f16", kind="step"),
        # the same of a large one
        _attend("step-128x4096", (32, 8, 128), 128, 4096, 16, "bf16", "bf16", by_head=False, kind="step"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.5 / hi)))))


def draw(rng):
    kind = rng.choice(["plan", "append", "attend", "attend", "attend", "step"])
    page = rng.choice(PAGES)
    if kind == "plan":
        rows = _log(rng, 1, 1000)
        return _plan(None, rows, _log(rng, 1, 8192), _log(rng, 1, 160000 // rows), page, rng.choice([0, 0, 2, 5]))
    heads, cache = rng.choice(HEADS), rng.choice(["f16", "bf16"])
    dtype, by_head = rng.choice([cache, cache, "f32"]), rng.random() < 0.5
    if kind == "append":
        return _append(None, heads, _log(rng, 1, 16384), page, cache, dtype, by_head)
    rows, skew = _log(rng, 1, 300), rng.choice([1, 1, 4])
    # at most half the largest case's positions (heads twice as many count twice), and what the plain form pads them to
    top = min(131071, 500000 * 16 // (rows * heads[0]))
    top = _log(rng, 1, top)
    window = rng.choice([0, 0, _log(rng, 1, 8000)])
    return _attend(None, heads, rows, top, page, cache, dtype, window, skew, by_head, kind)


# ---------------------------------------------------------------- inputs

def _cdiv(a, b):
    return -(-a // b)


def _lengths(case):
    """The rows' lengths, in no order: of four rows or more, one is idle; the longest is `top`."""
    n, top, skew = case["rows"], case["top"], case.get("skew", 1)
    got = [max(1, round(top * ((i + 1) / n) ** skew)) for i in range(n)]
    if n >= 4:
        got[0] = 0
    return got


def _news(case):
    """How many positions each row takes: every seventh none, the others 1 .. new."""
    n, new = case["rows"], case["new"]
    return [new if n == 1 else 0 if i % 7 == 6 else 1 + (new - 1) * i // (n - 1) for i in range(n)]


def _tokens(case):
    """Most tokens of a plan: the batch's, in whole blocks of 64 (a step's as it is)."""
    return case["rows"] if case["kind"] == "step" else _cdiv(sum(_news(case)), 64) * 64


def _int32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _pool(g, n_pages, case):
    dt = DTYPES[case["cache"]]
    hkv, hd, page = case["hkv"], case["hd"], case["page"]
    shape = (n_pages, hkv, page, hd) if case["by_head"] else (n_pages, page, hkv, hd)
    pools = []
    for _ in range(2):
        # a channel-wise spread of magnitudes, as rotated keys and values have
        spread = torch.exp(0.5 * torch.randn(hkv, 1, hd, generator=g, device="cuda"))
        pool = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        pool = pool if case["by_head"] else pool.transpose(1, 2)
        pools.append(pool.mul_(spread.to(dt)))
    return pools


def _tables(lens, width, n_pages, page, order):
    """[rows, width] of distinct pages in a shuffled order, the free stack behind them, and how many are free."""
    table = torch.zeros(len(lens), width, dtype=torch.int64)
    at = 0
    for i, n in enumerate(lens):
        m = _cdiv(n, page)
        table[i, :m] = order[at:at + m]
        at += m
    free = torch.zeros(n_pages, dtype=torch.int64)
    free[:n_pages - at] = order[at:]
    return table.to(torch.int32).cuda(), free.to(torch.int32).cuda(), _int32([n_pages - at])


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    kind, page = case["kind"], case["page"]
    s = {"case": case}
    if kind == "append":
        n = case["n"]
        n_pages = _cdiv(n, page) + 3
        s["k"], s["v"] = _pool(g, n_pages, case)
        # the new positions of a few requests, page by page, and every hundredth row of padding
        at = torch.arange(n)
        slots = torch.randperm(n_pages, generator=cpu)[at // page] * page + at % page
        slots[99::100] = -1
        s["slots"] = slots.to(torch.int32).cuda()
        s["rows"] = torch.randn(n, 2 * case["hkv"] * case["hd"], generator=g, device="cuda").to(DTYPES[case["dtype"]])
        return s
    rows = case["rows"]
    mix = torch.randperm(rows, generator=cpu).tolist()
    base = [_lengths(case)[i] for i in mix]
    if kind == "plan":
        news, fresh = _news(case), case["fresh"]
        s["n_new"] = _int32(news)
        # what the rows held before: up to 7 drafted positions more, and where a new request begins, an old one's
        lens = [b + (i * 5) % 8 for i, b in enumerate(base)]
        keep = [0 if fresh and i % fresh == fresh - 1 else b for i, b in enumerate(base)]
        after = [b + n for b, n in zip(keep, news)]
    elif kind == "step":
        s["n_new"] = _int32([1] * rows)
        keep, lens = [max(0, b - 1) for b in base], [max(0, b - 1) for b in base]
        after = [b + 1 for b in keep]
    else:
        lens = keep = after = base
    # room for any pairing of the rows with what they held and take
    more = _news(case) if kind == "plan" else [0]
    width = _cdiv(max(1, max(base)) + (max(7, max(more)) if kind == "plan" else 0), page)
    n_pages = sum(_cdiv(max(1, b) + (7 if kind == "plan" else 0), page) for b in base) + sum(_cdiv(n, page) for n in more) + 1
    s["tables"], s["free"], s["n_free"] = _tables(lens, width, n_pages, page, torch.randperm(n_pages, generator=cpu))
    s["lens"], s["keep"] = _int32(lens), _int32(keep)
    if kind != "plan":
        s["k"], s["v"] = _pool(g, n_pages, case)
        # the fused projection's output: q, k and v rows side by side
        s["rows"] = torch.randn(rows, (case["hq"] + 2 * case["hkv"]) * case["hd"], generator=g, device="cuda").to(DTYPES[case["dtype"]])
    return s


def _heads(state):
    """The rows' heads: (k, v) of an append, (q, k, v) else."""
    c = state["case"]
    x = state["rows"].unflatten(-1, (-1, c["hd"]))
    return x.split(([c["hq"]] if "hq" in c else []) + [c["hkv"], c["hkv"]], 1)


# ---------------------------------------------------------------- one pass

def _before(x):
    """Exclusive sums along the last dimension."""
    return x.cumsum(-1) - x


def _plain_plan(s):
    page, most = s["case"]["page"], _tokens(s["case"])
    table, lens, free, n_free = (s[k].long() for k in ("tables", "lens", "free", "n_free"))
    kept = torch.minimum(lens, s["keep"].long())
    new = kept + s["n_new"].long()
    held, stay, want = ((x + page - 1) // page for x in (lens, kept, new))
    j = torch.arange(table.shape[1], device=table.device)[None]
    pad = len(free)                                        # a place behind the stack, for entries that do not move
    free = torch.cat((free, free.new_zeros(1)))
    back, need = held - stay, want - stay
    top = n_free + back.sum()
    at = top - 1 - (_before(back)[:, None] + j - stay[:, None])
    at = torch.where((j >= stay[:, None]) & (j < held[:, None]), at, pad)
    free.scatter_(0, at.flatten(), table.flatten())
    at = top - 1 - (_before(need)[:, None] + j - stay[:, None])
    takes = (j >= stay[:, None]) & (j < want[:, None])
    table = torch.where(takes, free[torch.where(takes, at, pad)], table)
    s["tables"].copy_(table)
    s["free"].copy_(free[:-1])
    s["n_free"].copy_(top - need.sum())
    s["lens"].copy_(new)
    ends = s["n_new"].long().cumsum(0)
    t = torch.arange(most, device=table.device)
    row = torch.searchsorted(ends, t, right=True).clamp(max=len(ends) - 1)
    live = t < ends[-1]
    position = torch.where(live, kept[row] + t - (ends - s["n_new"])[row], 0)
    slots = torch.where(live, table[row, position // page] * page + position % page, -1)
    return slots.int(), position.int(), torch.cat((ends.new_zeros(1), ends)).int()


def _plain_append(s, k, v, slots):
    # (a row that goes nowhere is written over by another: the one that the first stored slot has anyway)
    slots = slots.long()
    first = torch.argmax((slots >= 0).to(torch.int32))
    row = torch.where(slots >= 0, torch.arange(len(slots), device=slots.device), first)
    page, at = slots[row] // s["case"]["page"], slots[row] % s["case"]["page"]
    for pool, x in ((s["k"], k), (s["v"], v)):
        pool[page, :, at] = x[row].to(pool.dtype)


def _plain_attend(s, q):
    c = s["case"]
    lens = s["lens"].long()
    k, v = (p[s["tables"].long()].transpose(1, 2).flatten(2, 3).float() for p in (s["k"], s["v"]))   # [rows, hkv, positions, hd]
    j = torch.arange(k.shape[2], device=k.device)[None]
    seen = j < lens[:, None]
    if c["window"]:
        seen &= j >= lens[:, None] - c["window"]
    qg = q.float().unflatten(1, (c["hkv"], -1))
    score = qg @ k.transpose(2, 3) / math.sqrt(c["hd"])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    o = p @ v / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.flatten(1, 2).to(q.dtype)


def run(state):
    c = state["case"]
    kind = c["kind"]
    if own:
        if "handles" not in state:   # what a program keeps: the batch's tables and the layer's cache, over its tensors, and its bound of a step's tokens
            import persistent_monokernel_gb300 as pm
            plans = kind in ("plan", "step")
            state["handles"] = (pm.PageTables.wrap(*(state[k] for k in ("tables", "lens", "free", "n_free")), c["page"]) if plans else None,
                                None if kind == "plan" else pm.PagedKVCache.wrap(state["k"], state["v"]), _tokens(c) if plans else 0)
        tables, cache, most = state["handles"]
        if kind == "append":
            k, v = _heads(state)
            cache.append(k, v, state["slots"])
            return state["k"], state["v"]
        if kind == "attend":
            return cache.attend(_heads(state)[0], state["tables"], state["lens"], window=c["window"])
        plan = tables.plan(state["n_new"], most, keep=state["keep"])
        if kind == "plan":
            return (*plan, state["tables"], state["lens"], state["free"], state["n_free"])
        q, k, v = _heads(state)
        cache.append(k, v, plan[0])
        return (*plan, cache.attend(q, state["tables"], state["lens"], window=c["window"]))
    if kind == "append":
        _plain_append(state, *_heads(state), state["slots"])
        return state["k"], state["v"]
    if kind == "attend":
        return _plain_attend(state, _heads(state)[0])
    plan = _plain_plan(state)
    if kind == "plan":
        return (*plan, state["tables"], state["lens"], state["free"], state["n_free"])
    q, k, v = _heads(state)
    _plain_append(state, k, v, plan[0])
    return (*plan, _plain_attend(state, q))


def work(case):
    kind = case["kind"]
    if kind == "append":
        n, values = case["n"] - case["n"] // 100, 2 * case["hkv"] * case["hd"]
        return {"bytes": 4 * case["n"] + n * values * (2 + DTYPES[case["dtype"]].itemsize), "flops": 0}
    rows, page = case["rows"], case["page"]
    if kind == "plan":
        news, tokens = _news(case), _tokens(case)
        # lens, keep, n_new, lens and offsets again; new pages off the stack and into the tables; slots and positions
        return {"bytes": 20 * rows + 8 * sum(_cdiv(n, page) for n in news) + 8 * tokens, "flops": 0}
    seen = [min(n, case["window"] or n) for n in _lengths(case)]
    if kind == "step":
        seen = [max(1, n) for n in seen]
    size, heads = DTYPES[case["dtype"]].itemsize, case["hq"] * case["hd"]
    b = sum(seen) * 4 * case["hkv"] * case["hd"] + 2 * rows * heads * size + 4 * sum(_cdiv(n, page) for n in seen) + 4 * rows
    if kind == "step":
        b += rows * (28 + 2 * case["hkv"] * case["hd"] * size)
    return {"bytes": b, "flops": 4 * sum(seen) * heads}


# ---------------------------------------------------------------- the same from the definition: lists, and 64 bits

def _exact_plan(state):
    """The plan by lists, one page at a time: (outputs, new tables as lists, new lengths)."""
    page = state["case"]["page"]
    table, lens, keep, n_new, free = (state[k].tolist() for k in ("tables", "lens", "keep", "n_new", "free"))
    top = state["n_free"].item()
    rows = range(len(lens))
    given = [table[i][j] for i in rows for j in range(_cdiv(min(lens[i], keep[i]), page), _cdiv(lens[i], page))]
    for p in reversed(given):
        free[top] = p
        top += 1
    slots, positions, offsets = [], [], [0]
    for i in rows:
        kept = min(lens[i], keep[i])
        for p in range(kept, kept + n_new[i]):
            if p % page == 0:
                top -= 1
                table[i][p // page] = free[top]
            slots.append(table[i][p // page] * page + p % page)
            positions.append(p)
        lens[i] = kept + n_new[i]
        offsets.append(len(slots))
    idle = _tokens(state["case"]) - len(slots)
    plan = [_int32(x) for x in (slots + [-1] * idle, positions + [0] * idle, offsets)]
    return plan, [_int32(x) for x in (table, lens, free, [top])]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "append":
        parts = _heads(s)
        for pool, x in ((s["k"], parts[0]), (s["v"], parts[1])):
            for t, slot in enumerate(s["slots"].tolist()):
                if slot >= 0:
                    pool[slot // case["page"], :, slot % case["page"]] = x[t]
        return s["k"], s["v"]
    plan = []
    if kind in ("plan", "step"):
        plan, after = _exact_plan(s)
        if kind == "plan":
            return (*plan, *after)
        s["tables"], s["lens"] = after[:2]
    q, k, v = (x.double() for x in _heads(s))
    page, group, hd = case["page"], case["hq"] // case["hkv"], case["hd"]
    out = torch.zeros(case["rows"], case["hq"], hd, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        at = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
        if not n:
            continue
        pages, place = s["tables"][i].long()[at // page], at % page
        for h in range(case["hkv"]):
            kk, vv = (pool[pages, h, place].double() for pool in (s["k"], s["v"]))
            if kind == "step":   # the new row, as the cache's type holds it
                kk[-1], vv[-1] = (x[i, h].to(s["k"].dtype).double() for x in (k, v))
            out[i, h * group:(h + 1) * group] = torch.softmax(q[i, h * group:(h + 1) * group] @ kk.T / math.sqrt(hd), -1) @ vv
    return (*plan, out) if plan else out
