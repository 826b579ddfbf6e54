"""The operators of the 4-bit KV cache: their cases and plain forms.

The cache of one layer holds K and V as 4-bit floats (E2M1: magnitudes 0, 0.5,
1, 1.5, 2, 3, 4, 6) with one 8-bit scale (E4M3) per 16 values of a row:
value = scale * e2m1.  codes are uint8 [n_kv_heads, max_seq, head_dim / 2]
(element 2i in the low nibble of byte i), scales uint8 [n_kv_heads, max_seq,
head_dim / 16].

  store    quantise n new rows of K and V into the cache and read them back:
           scale = E4M3(amax / 6), code = E2M1(x / scale), both to nearest even
  read     the values of n cached positions
  step     one decode step: the fused projection's k and v rows are appended and
           its q attends to the cache, the new position included
  attend   n queries at positions pos .. pos + n - 1 attend causally to a cache
           that holds them (a block of a prompt, or a few drafted tokens)

Query head h uses KV head h // (n_heads // n_kv_heads); with a window W > 0 the
query at position p sees max(0, p - W + 1) .. p.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# query heads, KV heads, head_dim of this repository's decoders (tiny, small, 2.3B, 8B shape), and two generic groupings
HEADS = [(4, 4, 64), (16, 4, 64), (20, 5, 128), (32, 8, 128), (8, 1, 128), (32, 4, 128)]


def _case(name, kind, heads, n, pos, dtype, window=0):
    """n new (or read, or querying) positions from pos on."""
    c = {"kind": kind, "hq": heads[0], "hkv": heads[1], "hd": heads[2], "n": n, "pos": pos, "dtype": dtype, "window": window}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token's rows: the smallest call, launches only
        _case("store-1", "store", (20, 5, 128), 1, 511, "f16"),
        # the batched prefill of a 512-token prompt
        _case("store-511", "store", (20, 5, 128), 511, 0, "f32"),
        # a session of the 2.3B decoder's long-context workload, in its cache's own type
        _case("store-32767", "store", (20, 5, 128), 32767, 0, "f16"),
        # a short session brought back
        _case("read-777", "read", (16, 4, 64), 777, 3, "bf16"),
        # a long one, for a program that works on the values
        _case("read-32768", "read", (32, 8, 128), 32768, 0, "f16"),
        # decoding right after a 512-token prompt
        _case("step-512", "step", (20, 5, 128), 1, 512, "f16"),
        # decoding at the 8B shape's prompt length, half-precision program, sliding window
        _case("step-2048-window", "step", (32, 8, 128), 1, 2048, "bf16", 1000),
        # decoding at 32k with the FP32 activations of this repository's decoders
        _case("step-32767", "step", (20, 5, 128), 1, 32767, "f32"),
        # the longest context: where the cache's bytes are all that counts
        _case("step-131071", "step", (32, 8, 128), 1, 131071, "f16"),
        # a few drafted tokens verified at once
        _case("attend-5-at-4097", "attend", (16, 4, 64), 5, 4097, "f16"),
        # a whole prompt, FP32 activations
        _case("attend-511-at-0", "attend", (20, 5, 128), 511, 0, "f32"),
        # a block of a long prompt, far into it: the largest
        _case("attend-1024-at-31744", "attend", (20, 5, 128), 1024, 31744, "f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.5 / hi)))))


def draw(rng):
    kind = rng.choice(["store", "read", "step", "attend", "attend"])
    hq, hkv, hd = heads = rng.choice(HEADS)
    dtype = rng.choice(sorted(DTYPES))
    if kind in ("store", "read"):
        return _case(None, kind, heads, _log(rng, 1, 32767), rng.randrange(0, 4000), dtype)
    window = rng.choice([0, 0, _log(rng, 1, 8000)])
    if kind == "step":
        return _case(None, kind, heads, 1, _log(rng, 1, 131071), dtype, window)
    n = _log(rng, 2, 1024)
    top = min(31744, 1024 * 32768 * 20 // (n * hq) - n)
    # fp32 queries cost twice the products: half the positions at most
    pos = _log(rng, 1, top // 2 if dtype == "f32" else top) - 1
    return _case(None, kind, heads, n, pos, dtype, window)


# ---------------------------------------------------------------- inputs

def _quantise(x):
    """FP32 [.., hd] to (codes, scales) bytes."""
    b = x.float().unflatten(-1, (-1, 16))
    s8 = (b.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    a = torch.where(s > 0, b.abs() / s, torch.zeros_like(b))
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    c = (c | ((b < 0) & (s > 0)).to(torch.uint8) << 3).flatten(-2)
    return c[..., 0::2] | c[..., 1::2] << 4, s8.view(torch.uint8)


def _values(codes, scales):
    """(codes, scales) bytes to FP32 [.., hd]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    v = mags[(c & 7).long()] * (1 - 2 * (c >> 3).float())
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _capacity(case):
    """Positions of the cache: room behind the last one, in whole blocks of 256."""
    return (case["pos"] + case["n"] + 255) // 256 * 256


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    hq, hkv, hd, n = case["hq"], case["hkv"], case["hd"], case["n"]
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    cap = _capacity(case)
    if case["kind"] == "store":
        parts = [torch.zeros(hkv, cap, w, dtype=torch.uint8, device="cuda") for w in (hd // 2, hd // 16)] * 2
        parts = [p.clone() for p in parts]
    else:
        # a channel-wise spread of magnitudes, as rotated keys and values have
        spread = torch.exp(0.5 * normal(2, hkv, 1, hd))
        parts = [t for i in range(2) for t in _quantise(normal(hkv, cap, hd) * spread[i])]
    # the fused projection's output: q, k and v rows side by side
    qkv = normal(n, (hq + 2 * hkv) * hd).to(dt)
    return {"case": case, "parts": parts, "qkv": qkv}


def _split(state):
    c = state["case"]
    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    return state["qkv"].unflatten(-1, (-1, hd)).split((hq, hkv, hkv), 1)


# ---------------------------------------------------------------- one pass

def _plain_append(state):
    c = state["case"]
    _, k, v = _split(state)
    for x, codes, scales in ((k, *state["parts"][:2]), (v, *state["parts"][2:])):
        qc, qs = _quantise(x.transpose(0, 1))
        codes[:, c["pos"]:c["pos"] + c["n"]] = qc
        scales[:, c["pos"]:c["pos"] + c["n"]] = qs


def _plain_read(state, lo, hi):
    p = state["parts"]
    return [_values(p[i][:, lo:hi], p[i + 1][:, lo:hi]) for i in (0, 2)]


def _seen(case, lo, hi, device):
    """[n, hi - lo]: which positions each query sees."""
    at = torch.arange(case["pos"], case["pos"] + case["n"], device=device)[:, None]
    j = torch.arange(lo, hi, device=device)
    return (j <= at) & (j > at - case["window"]) if case["window"] else j <= at


def _first(case):
    """The first position that any query sees."""
    return max(0, case["pos"] - case["window"] + 1) if case["window"] else 0


def _plain_attend(state):
    c = state["case"]
    q = _split(state)[0].float()
    lo, hi = _first(c), c["pos"] + c["n"]
    k, v = _plain_read(state, lo, hi)
    qg = q.unflatten(1, (c["hkv"], -1)).permute(1, 2, 0, 3).flatten(1, 2)           # [hkv, group * n, hd]
    s = (qg @ k.transpose(1, 2) / math.sqrt(c["hd"])).unflatten(1, (-1, c["n"]))
    s = s.masked_fill(~_seen(c, lo, hi, q.device), -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = (p / p.sum(-1, keepdim=True)).flatten(1, 2) @ v
    o = o.unflatten(1, (-1, c["n"])).permute(2, 0, 1, 3).flatten(1, 2)
    return o.to(DTYPES[c["dtype"]])


def run(state):
    c = state["case"]
    kind, n, pos = c["kind"], c["n"], c["pos"]
    if own:
        cache = state.get("cache")
        if cache is None:   # the handle that a program keeps: the cache's four tensors
            import persistent_monokernel_gb300 as pm
            cache = state["cache"] = pm.KV4Cache.wrap(*state["parts"])
        if kind == "read":
            return cache.read(pos, n, DTYPES[c["dtype"]])
        q, k, v = _split(state)
        if kind == "attend":
            return cache.attend(q, pos, window=c["window"])
        cache.append(k, v, pos)
        return cache.read(pos, n, DTYPES[c["dtype"]]) if kind == "store" else cache.attend(q, pos, window=c["window"])
    if kind in ("store", "step"):
        _plain_append(state)
    if kind in ("store", "read"):
        return tuple(x.transpose(0, 1).to(DTYPES[c["dtype"]]).contiguous() for x in _plain_read(state, pos, pos + n))
    return _plain_attend(state)


def work(case):
    hq, hkv, hd, n, pos, w = (case[k] for k in ("hq", "hkv", "hd", "n", "pos", "window"))
    size = torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
    packed, rows = 2 * hkv * (hd // 2 + hd // 16), 2 * n * hkv * hd * size   # bytes of a cached position; of n plain ones
    if case["kind"] == "store":
        return {"bytes": 2 * rows + n * packed, "flops": 0}
    if case["kind"] == "read":
        return {"bytes": rows + n * packed, "flops": 0}
    pairs = sum(min(p + 1, w or p + 1) for p in range(pos, pos + n))
    b = (pos + n - _first(case)) * packed + 2 * n * hq * hd * size
    if case["kind"] == "step":
        b += rows
    return {"bytes": b, "flops": 4 * pairs * hq * hd}


# ---------------------------------------------------------------- the same from the definition, in 64 bits

def _field(bits, ebits, mbits, bias):
    """Minifloats of `ebits` exponent and `mbits` mantissa bits, as integers, to FP64."""
    bits = bits.int()
    e, m = bits >> mbits & (1 << ebits) - 1, (bits & (1 << mbits) - 1).double() / (1 << mbits)
    mag = torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * torch.exp2((e - bias).double()))
    return torch.where(bits >> (ebits + mbits) & 1 == 1, -mag, mag)


def _exact_values(codes, scales):
    """(codes, scales) bytes to FP64 [.., hd], from the formats' fields."""
    v = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    v[..., 0::2], v[..., 1::2] = _field(codes & 15, 2, 1, 1), _field(codes >> 4, 2, 1, 1)
    return v * _field(scales, 4, 3, 7).repeat_interleave(16, -1)


def _nearest_even(x, grid):
    """Index of the entry of the ascending `grid` nearest to x >= 0, halfway cases to the even index."""
    i = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    below, above = x - grid[i - 1], grid[i] - x
    up = (above < below) | ((above == below) & (i % 2 == 0))
    return torch.where(up, i, i - 1)


def _exact_round(x):
    """FP64 [.., hd] to the values that its 4-bit form stands for."""
    b = x.double().unflatten(-1, (-1, 16))
    scale_grid = _field(torch.arange(127, device=x.device), 4, 3, 7)
    mag_grid = _field(torch.arange(8, device=x.device), 2, 1, 1)
    s = scale_grid[_nearest_even(b.abs().amax(-1, keepdim=True) / 6, scale_grid)]
    a = torch.where(s > 0, b.abs() / s, torch.zeros_like(b))
    return (torch.sign(b) * s * mag_grid[_nearest_even(a, mag_grid)]).flatten(-2)


def exact(case, seed):
    state = prepare(case, seed)
    n, pos, hkv, hd = case["n"], case["pos"], case["hkv"], case["hd"]
    q, k, v = _split(state)
    kc, ks, vc, vs = state["parts"]
    if case["kind"] == "store":
        return tuple(_exact_round(x) for x in (k, v))
    if case["kind"] == "read":
        return tuple(_exact_values(a[:, pos:pos + n], b[:, pos:pos + n]).transpose(0, 1).contiguous() for a, b in ((kc, ks), (vc, vs)))
    out = torch.empty(n, case["hq"], hd, dtype=torch.float64, device="cuda")
    group = case["hq"] // hkv
    at = pos + torch.arange(n, device="cuda")
    for h in range(case["hq"]):   # one head at a time, every position of the cache
        kk, vv = (_exact_values(a[h // group, :pos + n], b[h // group, :pos + n]) for a, b in ((kc, ks), (vc, vs)))
        if case["kind"] == "step":
            kk[pos:], vv[pos:] = _exact_round(k[:, h // group]), _exact_round(v[:, h // group])
        s = q[:, h].double() @ kk.T / math.sqrt(hd)
        j = torch.arange(pos + n, device="cuda")
        hidden = j[None] > at[:, None]
        if case["window"]:
            hidden |= j[None] <= at[:, None] - case["window"]
        out[:, h] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ vv
    return out
