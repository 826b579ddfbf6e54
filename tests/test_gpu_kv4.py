"""The 4-bit KV cache operators on the GPU against their definition in 64 bits."""
import math

import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def pm():
    import persistent_monokernel_gb300 as pm
    from persistent_monokernel_gb300 import build
    build.build()
    return pm


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def filled(pm, hkv, hd, cap, seed, spread=True):
    """A cache of random rows (quantised by the reference) and its values in FP64."""
    g = gen(seed)
    parts, vals = [], []
    for _ in range(2):
        x = torch.randn(hkv, cap, hd, generator=g, device="cuda")
        if spread:
            x = x * torch.exp(0.5 * torch.randn(hkv, 1, hd, generator=g, device="cuda"))
        c, s = ref.quantise(x)
        parts += [c, s]
        vals.append(ref.values(c, s))
    return pm.KV4Cache.wrap(*parts), vals


def check(out, want, bound):
    assert torch.isfinite(out).all()
    err = (out.double() - want).abs()
    worst = (err / bound).max().item()
    assert worst <= 1, f"{worst:.3g} times the bound"


# ---------------------------------------------------------------- append and read

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hkv,hd,n,pos", [(1, 64, 1, 0), (5, 128, 1, 300), (4, 64, 37, 5), (3, 128, 129, 1), (8, 128, 2, 254)])
@pytest.mark.parametrize("size", [1e-3, 0.02, 1.0, 300.0, 5000.0])
def test_append_stores_the_nearest_codes_and_leaves_the_other_rows(pm, dtype, hkv, hd, n, pos, size):
    g = gen(n + hd)
    x = [(torch.randn(n, hkv, hd, generator=g, device="cuda") * size).to(dtype) for _ in range(2)]
    x[0][0, 0, :16] = 0                                   # an empty block
    cache = pm.KV4Cache(hkv, hd, 430)
    parts = (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)
    for p in parts:
        p.fill_(0x5a)
    cache.append(x[0], x[1], pos)
    for i, t in enumerate(x):
        c, s = ref.quantise(t)
        for got, want in ((parts[2 * i], c), (parts[2 * i + 1], s)):
            assert torch.equal(got[:, pos:pos + n], want.transpose(0, 1))
            assert (got[:, :pos] == 0x5a).all() and (got[:, pos + n:] == 0x5a).all()


def test_append_takes_ties_to_even(pm):
    # scale 1 (largest magnitude 6): every half-way value and its neighbours
    vals = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 0]
    rows = [vals]
    for step in (1 + 2.0 ** -10, 1 - 2.0 ** -10):
        rows.append([6] + [v * step for v in vals[1:]])
    # scales half-way between two E4M3 values: 1.0625 * 6 and 1.1875 * 6
    rows += [[6.375] + [1.0] * 15, [7.125] + [1.0] * 15]
    x = torch.tensor(rows, dtype=torch.float16, device="cuda").repeat(1, 4).unsqueeze(1).contiguous()
    cache = pm.KV4Cache(1, 64, len(rows))
    cache.append(x, x, 0)
    c, s = ref.quantise(x)
    assert torch.equal(cache.k_codes[0], c[:, 0]) and torch.equal(cache.v_scales[0], s[:, 0])
    assert cache.k_scales[0, 3, 0].item() == 0x38 and cache.k_scales[0, 4, 0].item() == 0x3a   # to even


def test_append_of_non_finite_values_stays_finite(pm):
    x = torch.randn(4, 2, 64, generator=gen(0), device="cuda").half()
    x[0, 0, 3], x[1, 1, 20], x[2, 0, 40], x[3, 1, :16] = math.nan, math.inf, -math.inf, math.nan
    for t in (x, x.float(), x.bfloat16()):
        cache = pm.KV4Cache(2, 64, 8)
        cache.append(t, t, 2)
        c, s = ref.quantise(t)
        assert torch.equal(cache.k_codes[:, 2:6], c.transpose(0, 1)) and torch.equal(cache.v_scales[:, 2:6], s.transpose(0, 1))
        k, _ = cache.read(2, 4, torch.float32)
        assert torch.isfinite(k).all() and k[1, 1, 20] == 2688 and k[2, 0, 40] == -2688 and k[0, 0, 3] == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hkv,hd,n,pos", [(1, 64, 1, 9), (5, 128, 333, 17), (2, 64, 64, 0)])
def test_read_returns_the_values_exactly(pm, dtype, hkv, hd, n, pos):
    g = gen(7)
    cap = pos + n + 3
    codes = [torch.randint(0, 256, (hkv, cap, hd // 2), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    scales = [torch.randint(0, 127, (hkv, cap, hd // 16), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    cache = pm.KV4Cache.wrap(codes[0], scales[0], codes[1], scales[1])
    got = cache.read(pos, n, dtype)
    for t, c, s in zip(got, codes, scales):
        assert t.dtype == dtype and t.shape == (n, hkv, hd)
        assert torch.equal(t.double(), ref.values(c, s)[:, pos:pos + n].transpose(0, 1))
    # into tensors of the caller: a [heads, n, hd] one and a slice of a wider one
    wide = torch.full((n, 3 * hkv, hd), 7, dtype=dtype, device="cuda")
    turned = torch.empty(hkv, n, hd, dtype=dtype, device="cuda")
    cache.read(pos, n, out=(turned.transpose(0, 1), wide[:, hkv:2 * hkv]))
    assert torch.equal(turned.transpose(0, 1), got[0]) and torch.equal(wide[:, hkv:2 * hkv], got[1])
    assert (wide[:, :hkv] == 7).all() and (wide[:, 2 * hkv:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_from_a_fused_projection_and_a_transposed_tensor(pm, dtype):
    g = gen(3)
    qkv = torch.randn(19, (4 + 2 * 2) * 64, generator=g, device="cuda").to(dtype).unflatten(-1, (-1, 64))
    _, k, v = qkv.split((4, 2, 2), 1)
    a, b, c = (pm.KV4Cache(2, 64, 32) for _ in range(3))
    a.append(k, v, 4)
    b.append(k.contiguous(), v.contiguous(), 4)
    c.append(k.transpose(0, 1).contiguous().transpose(0, 1), v.transpose(0, 1).contiguous().transpose(0, 1), 4)
    for other in (b, c):
        assert torch.equal(a.k_codes, other.k_codes) and torch.equal(a.v_scales, other.v_scales)
        assert torch.equal(a.v_codes, other.v_codes) and torch.equal(a.k_scales, other.k_scales)


# ---------------------------------------------------------------- attention

HEADS = [(4, 4, 64), (16, 4, 64), (20, 5, 128), (8, 1, 128), (3, 1, 64), (24, 2, 128)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv,hd", HEADS)
@pytest.mark.parametrize("n,pos", [(1, 0), (1, 1), (1, 31), (1, 1000), (1, 5000), (2, 63), (5, 700), (3, 0)])
def test_attend_few_rows(pm, dtype, hq, hkv, hd, n, pos):
    cache, (k, v) = filled(pm, hkv, hd, pos + n + 5, pos + hd)
    q = torch.randn(n, hq, hd, generator=gen(n), device="cuda").to(dtype)
    check(cache.attend(q, pos), *ref.attention(q, k, v, pos, pos + n, 0, 0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv,hd", [(16, 4, 64), (20, 5, 128), (8, 1, 128), (24, 2, 128)])
@pytest.mark.parametrize("n,pos", [(33, 0), (64, 64), (129, 0), (200, 1000), (511, 1), (130, 4000), (1024, 3)])
def test_attend_blocks(pm, dtype, hq, hkv, hd, n, pos):
    cache, (k, v) = filled(pm, hkv, hd, pos + n + 5, pos + hd)
    q = torch.randn(n, hq, hd, generator=gen(n), device="cuda").to(dtype)
    check(cache.attend(q, pos), *ref.attention(q, k, v, pos, pos + n, 0, 0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv,hd,n,pos,window", [
    (32, 8, 128, 700, 0, 0), (32, 8, 64, 1100, 130, 0), (15, 5, 64, 1400, 9, 0), (24, 8, 128, 900, 1, 200),   # more tiles than SMs
    (40, 1, 128, 1, 3000, 0), (33, 1, 64, 1, 20000, 0), (34, 1, 64, 1, 127, 0), (80, 2, 128, 1, 9000, 5000),  # one token
    (9, 1, 64, 60, 7000, 0), (12, 4, 128, 90, 6000, 0), (35, 5, 64, 77, 2500, 1111)])                         # odd groups, cut tiles
def test_attend_many_tiles_and_wide_groups(pm, dtype, hq, hkv, hd, n, pos, window):
    cache, (k, v) = filled(pm, hkv, hd, pos + n, pos + hd)
    q = torch.randn(n, hq, hd, generator=gen(n), device="cuda").to(dtype)
    check(cache.attend(q, pos, window=window), *ref.attention(q, k, v, pos, pos + n, window, 0))


def test_attend_after_calls_of_the_same_shape_elsewhere(pm):
    """The same rows at short, long and short contexts again: scratch is asked for by shape, the need depends on more."""
    cache, (k, v) = filled(pm, 2, 64, 31000, 8)
    for n in (1, 20, 200, 1000):
        q = torch.randn(n, 8, 64, generator=gen(n), device="cuda").half()
        for pos, window in ((5, 0), (29000, 0), (64, 0), (29500, 300), (12000, 0), (0, 0)):
            check(cache.attend(q, pos, window=window), *ref.attention(q, k, v, pos, pos + n, window, 0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,bad", [(3, 1), (150, 40), (2000, 777)])
def test_a_row_that_is_not_finite_stays_by_itself(pm, dtype, n, bad):
    """q has to be finite; a padded row that is not may spoil its own output only."""
    cache, (k, v) = filled(pm, 2, 128, 2850 + n, 8)
    q = torch.randn(n, 4, 128, generator=gen(n), device="cuda").to(dtype)
    want, bound = ref.attention(q, k, v, 2700, 2700 + n, 0, 0)
    rest = [i for i in range(n) if i != bad]
    for value in (math.nan, math.inf, -math.inf):
        q[bad, :, ::3] = value
        check(cache.attend(q, 2700)[rest], want[rest], bound[rest])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,pos,length,window", [
    (1, 900, 901, 1), (1, 900, 901, 17), (1, 900, 901, 900), (1, 900, 901, 901), (1, 900, 901, 5000),
    (7, 900, 907, 3), (7, 900, 907, 64), (150, 700, 850, 40), (300, 0, 300, 33), (260, 3000, 3260, 1000),
    (200, 100, 150, 0), (200, 100, 50, 0), (4, 10, 3, 0), (1300, 700, 2000, 40), (1500, 0, 1500, 33), (1400, 3000, 4400, 1000),
    (1300, 100, 1200, 0), (1300, 100, 50, 0), (1300, 100, 700, 90)])
def test_attend_windows_and_lengths(pm, dtype, n, pos, length, window):
    cache, (k, v) = filled(pm, 2, 128, max(length, pos + n), 5)
    q = torch.randn(n, 8, 128, generator=gen(n), device="cuda").to(dtype)
    check(cache.attend(q, pos, length=length, window=window), *ref.attention(q, k, v, pos, length, window, 0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
def test_rows_that_see_nothing_are_zero(pm, dtype, hd):
    cache, (k, v) = filled(pm, 2, hd, 400, 1)
    for n in (1, 6, 300, 1600):
        q = torch.randn(n, 8, hd, generator=gen(n), device="cuda").to(dtype)
        # an empty cache; a window past the last position for some rows, for all of them
        assert (cache.attend(q, 0, length=0) == 0).all()
        out = cache.attend(q, 90, length=100, window=20)
        check(out, *ref.attention(q, k, v, 90, 100, 20, 0))
        assert (out[30:] == 0).all()
        assert (cache.attend(q, 500, length=400, window=50) == 0).all()
        assert cache.attend(q[:0], 0).shape == (0, 8, hd)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 4, 150, 2000])
def test_positions_that_no_row_sees_do_not_count(pm, dtype, n):
    """Scales that stand for NaN (never written by append) before the window and behind the last position."""
    cache, (k, v) = filled(pm, 2, 64, 550 + n, 9)
    pos, window = 333, 100
    q = torch.randn(n, 4, 64, generator=gen(n), device="cuda").to(dtype)
    want = ref.attention(q, k, v, pos, pos + n, window, 0)
    clean = cache.attend(q, pos, window=window)
    for s in (cache.k_scales, cache.v_scales):
        s[:, :pos - window + 1] = 0x7f
        s[:, pos + n:] = 0x7f
    out = cache.attend(q, pos, window=window)
    check(out, *want)
    assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 6, 140, 1300])
@pytest.mark.parametrize("size,scale", [(30.0, 0.0), (1.0, 2.5), (1.0, -0.3), (1e-6, 1e5), (1000.0, 1e-3), (0.0, 0.0)])
def test_attend_scales_and_sizes_of_q(pm, dtype, n, size, scale):
    cache, (k, v) = filled(pm, 2, 128, 460 + n, 2)
    q = (torch.randn(n, 8, 128, generator=gen(n), device="cuda") * size).to(dtype)
    check(cache.attend(q, 400, scale=scale), *ref.attention(q, k, v, 400, 400 + n, 0, scale))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 140, 2500])
def test_q_beyond_the_range_of_fp16(pm, dtype, n):
    cache, (k, v) = filled(pm, 2, 64, 460 + n, 2)
    for size in (1e8, 1e-12, 1e30):
        q = (torch.randn(n, 4, 64, generator=gen(n), device="cuda") * size).to(dtype)
        check(cache.attend(q, 400, scale=1 / size / 8), *ref.attention(q, k, v, 400, 400 + n, 0, 1 / size / 8))


@pytest.mark.parametrize("n", [1, 5, 140, 1300])
def test_attend_layouts(pm, n):
    cache, _ = filled(pm, 2, 128, 560 + n, 4)
    qkv = torch.randn(n, 12, 128, generator=gen(n), device="cuda").half()
    q = qkv[:, :8]
    want = cache.attend(q.contiguous(), 500)
    assert torch.equal(cache.attend(q, 500), want)
    assert torch.equal(cache.attend(q.transpose(0, 1).contiguous().transpose(0, 1), 500), want)
    wide = torch.full((n, 20, 128), 3.0, dtype=torch.float16, device="cuda")
    assert cache.attend(q, 500, out=wide[:, 4:12]).data_ptr() == wide[:, 4:12].data_ptr()
    assert torch.equal(wide[:, 4:12], want) and (wide[:, :4] == 3).all() and (wide[:, 12:] == 3).all()
    turned = torch.empty(8, n, 128, dtype=torch.float16, device="cuda")
    cache.attend(q, 500, out=turned.transpose(0, 1))
    assert torch.equal(turned.transpose(0, 1), want)
    # every row the same: a broadcast query
    same = q[:1].expand(n, 8, 128)
    assert torch.equal(cache.attend(same, 500), cache.attend(same.contiguous(), 500))


@pytest.mark.parametrize("n", [1, 5, 140])
def test_the_same_call_gives_the_same_bits(pm, n):
    cache, _ = filled(pm, 5, 128, 5000, 4)
    q = torch.randn(n, 20, 128, generator=gen(n), device="cuda")
    first = cache.attend(q, 4800)
    for _ in range(5):
        assert torch.equal(cache.attend(q, 4800), first)


def test_long_context(pm):
    """131,072 positions, 8 KV heads: row offsets of 67 MB; one head of a 20-million position cache: offsets past 2^30."""
    cache, (k, v) = filled(pm, 8, 128, 131072, 11)
    q = torch.randn(1, 8, 128, generator=gen(1), device="cuda").half()
    check(cache.attend(q, 131071), *ref.attention(q, k, v, 131071, 131072, 0, 0))


def test_offsets_past_32_bits(pm):
    """A cache whose code bytes pass 2^32: the last head's last rows."""
    hkv, hd, cap = 70, 128, 1 << 20
    cache = pm.KV4Cache(hkv, hd, cap)
    assert cache.k_codes.numel() > 1 << 32
    g = gen(5)
    n = 200
    k, v = (torch.randn(n, hkv, hd, generator=g, device="cuda").half() for _ in range(2))
    cache.append(k, v, cap - n)
    got = cache.read(cap - n, n)
    want = [ref.values(*ref.quantise(t)) for t in (k, v)]
    assert all(torch.equal(a.double(), b) for a, b in zip(got, want))
    for rows in (1, 150):
        q = torch.randn(rows, hkv, hd, generator=g, device="cuda").half()
        kk, vv = (t.transpose(0, 1) for t in want)
        # the window covers just what was written: the reference's position 0 is the cache's cap - n
        out = cache.attend(q, cap - rows, window=n - rows + 1)
        check(out, *ref.attention(q, kk, vv, n - rows, n, n - rows + 1, 0))


# ---------------------------------------------------------------- together, on streams and in graphs

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv,hd,window", [(20, 5, 128, 0), (16, 4, 64, 30)])
def test_a_prompt_then_decode_steps(pm, dtype, hq, hkv, hd, window):
    """A prompt in two blocks, then single tokens, each appended and attended to from one fused projection."""
    g = gen(1)
    cache = pm.KV4Cache(hkv, hd, 256)
    k64 = torch.zeros(hkv, 0, hd, dtype=torch.float64, device="cuda")
    v64 = k64
    pos = 0
    for n in (90, 41, 1, 1, 1, 4, 1):
        q, k, v = torch.randn(n, hq + 2 * hkv, hd, generator=g, device="cuda").to(dtype).split((hq, hkv, hkv), 1)
        k64, v64 = (torch.cat((a, ref.values(*ref.quantise(b)).transpose(0, 1)), 1) for a, b in ((k64, k), (v64, v)))
        cache.append(k, v, pos)
        check(cache.attend(q, pos, window=window), *ref.attention(q, k64, v64, pos, pos + n, window, 0))
        pos += n


def test_captured_and_replayed(pm):
    """append + attend in a CUDA graph, replayed with new inputs in the same buffers, beside eager calls."""
    cache, _ = filled(pm, 5, 128, 2100, 3)
    qkv = torch.randn(1, 30, 128, generator=gen(0), device="cuda").half()
    block = torch.randn(150, 20, 128, generator=gen(1), device="cuda").half()
    q, k, v = qkv.split((20, 5, 5), 1)
    cache.append(k, v, 2000)
    cache.attend(q, 2000), cache.attend(block, 1850)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.append(k, v, 2000)
            outs = (cache.attend(q, 2000), cache.attend(block, 1850))
        graphs.append((g, outs))
    for seed in range(3):
        qkv.copy_(torch.randn(1, 30, 128, generator=gen(10 + seed), device="cuda"))
        for g, outs in graphs:
            g.replay()
        cache.append(k, v, 2000)
        want = (cache.attend(q, 2000), cache.attend(block, 1850))
        for g, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_streams_at_once(pm):
    """Reads of one cache on two streams share nothing."""
    cache, _ = filled(pm, 5, 128, 4000, 3)
    qs = [torch.randn(n, 20, 128, generator=gen(n), device="cuda") for n in (1, 3, 140)]
    want = [cache.attend(q, 3800) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s in streams:
            got += [(i, cache.attend(q, 3800, stream=s)) for i, q in enumerate(qs)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in got)


def test_threads_on_one_stream(pm):
    """Calls that need scratch from several threads: what one lets go of before its launch would be another's."""
    from concurrent.futures import ThreadPoolExecutor
    cache, _ = filled(pm, 8, 128, 40000, 3)
    qs = [torch.randn(n, h, 128, generator=gen(n), device="cuda").half() for n, h in ((1, 8), (140, 32), (1, 16), (3, 8))]
    want = [cache.attend(q, 39000) for q in qs]

    def work(i):
        return all([torch.equal(cache.attend(qs[i], 39000), want[i]) for _ in range(100)])

    with ThreadPoolExecutor(4) as ex:
        assert all(ex.map(work, range(4)))


def test_what_is_no_tensor_or_no_number(pm):
    cache = pm.KV4Cache(2, 64, 32)
    x, q = (torch.randn(4, h, 64, device="cuda").half() for h in (2, 8))
    for call in (lambda: cache.append(None, x, 0), lambda: cache.append(x, [1], 0), lambda: cache.attend(3, 0),
                 lambda: cache.append(x[0], x, 0), lambda: cache.attend(q[0, 0], 0), lambda: cache.attend(q, 0, out=x),
                 lambda: cache.read(0, 4, out=(x, None)), lambda: cache.read(0, 4, out=(x,)), lambda: cache.attend(q.to_sparse(), 0),
                 lambda: cache.attend(q.double(), 0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cache.append(x, x, None), lambda: cache.append(x, x, 0.5), lambda: cache.attend(q, None),
                 lambda: cache.attend(q, 0, window=None), lambda: cache.attend(q, 0, scale="1"), lambda: cache.read("0", 1),
                 lambda: cache.attend(q, 0, length=1.0)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: cache.attend(q, 0, out=q.float()), lambda: cache.read(0, 2 ** 31 - 1), lambda: cache.read(2 ** 31 - 1, 2 ** 31 - 1), lambda: cache.attend(q, 2 ** 31 - 1),
                 lambda: cache.append(x.expand(4, 2, 64)[:1].expand(33, 2, 64), x[:1].expand(33, 2, 64), 0)):
        with pytest.raises(pm.LFError):
            call()
    assert (cache.k_codes == 0).all()
    # positions as NumPy and torch integers, results in tensors that the caller keeps
    i = torch.tensor(3)
    cache.append(x, x, i)
    k, v = cache.read(i, 4)
    assert cache.read(3, 4, out=(k, v))[1] is v and torch.equal(k, v)
    out = torch.empty_like(q)
    assert cache.attend(q, i, out=out) is out and torch.equal(out, cache.attend(q, 3))


def test_calls_keep_no_memory(pm):
    """References and scratch go with the call, refused ones too."""
    import gc
    import sys
    cache = filled(pm, 8, 128, 40000, 3)[0]
    q = torch.randn(1, 8, 128, device="cuda").half()
    out, row = torch.empty_like(q), torch.empty_like(q)
    cache.attend(q, 39000)
    gc.collect()                                          # of earlier tests
    before, refs = torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in (q, out, row)]
    for _ in range(20):
        cache.attend(q, 39000)
        cache.attend(q, 39000, out=out)
        cache.read(39000, 1), cache.read(0, 1, out=(out, row)), cache.append(q, q, 39999)
        for call in (lambda: cache.attend(q, 39000, window=-1), lambda: cache.attend(q, 39000, out=q), lambda: cache.read(0, 2, out=(out, row)),
                     lambda: cache.attend(q, 39000, out=out[0]), lambda: cache.append(q, q, 40000), lambda: cache.attend(q, 2 ** 40, out=out)):
            with pytest.raises((pm.LFError, ValueError)):
                call()
    assert torch.cuda.memory_allocated() == before and [sys.getrefcount(t) for t in (q, out, row)] == refs


def test_the_first_calls_of_a_process_may_be_captured():
    """Kernels that no call has loaded yet, recorded at once."""
    import subprocess
    import sys

    from conftest import ROOT
    code = """
import torch, persistent_monokernel_gb300 as pm
cache = pm.KV4Cache(2, 128, 6000)
k = torch.randn(5000, 2, 128, device="cuda").half()
q, b = torch.randn(1, 8, 128, device="cuda").half(), torch.randn(100, 8, 128, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    cache.append(k, k, 0)
    outs = cache.attend(q, 4999), cache.attend(b, 4900), cache.read(7, 9)[0]
g.replay()
torch.cuda.synchronize()
assert cache.sync() == 0
want = cache.attend(q, 4999), cache.attend(b, 4900), cache.read(7, 9)[0]
assert all(torch.equal(x, y) and y.abs().sum() > 0 for x, y in zip(outs, want))
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, timeout=300)


def test_refusals_in_python(pm):
    cache = pm.KV4Cache(2, 64, 32)
    x = torch.randn(4, 2, 64, device="cuda").half()
    q = torch.randn(4, 8, 64, device="cuda").half()
    for bad in (x.cpu(), x[:, :1], x[:, :, :32], x.double(), x.transpose(1, 2).contiguous().transpose(1, 2), x[:3]):
        with pytest.raises(ValueError):
            cache.append(x, bad, 0)
    odd = torch.empty(4 * 2 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(4, 2, 64)
    for call in (lambda: cache.append(x, odd, 0), lambda: cache.append(x, x, 30), lambda: cache.append(x, x, -1),
                 lambda: cache.append(x, x.float(), 0), lambda: cache.read(30, 4), lambda: cache.read(0, -1),
                 lambda: cache.read(0, 4, out=(x, x[:1].expand(4, 2, 64))), lambda: cache.attend(q, 30),
                 lambda: cache.attend(q, 0, length=33), lambda: cache.attend(q, -1), lambda: cache.attend(q, 0, window=-1),
                 lambda: cache.attend(q, 0, scale=math.inf), lambda: cache.attend(q[:, :3], 0),
                 lambda: cache.attend(q, 0, out=q)):
        with pytest.raises(pm.LFError):
            call()
    for call in (lambda: cache.append(x, x, 2 ** 32), lambda: cache.read(2 ** 32, 1), lambda: cache.attend(q, 2 ** 32),
                 lambda: cache.read(0, 4, torch.float64), lambda: cache.attend(q, 0, out=q[:3]),
                 lambda: cache.attend(q, 0, out=q.float().half()[..., :32])):
        with pytest.raises((ValueError, pm.LFError)):
            call()
    assert cache.sync() == 0
    assert (cache.k_codes == 0).all() and (cache.v_scales == 0).all()


def test_on_a_stream_that_is_not_the_current_one(pm):
    """Inputs made, appended, attended to and read on a side stream, while the current one is busy."""
    s = torch.cuda.Stream()
    cache, _ = filled(pm, 5, 128, 9000, 2)
    qkv = torch.randn(1, 30, 128, generator=gen(1), device="cuda").half()
    q, k, v = qkv.split((20, 5, 5), 1)
    cache.append(k, v, 8990)
    want, row = cache.attend(q, 8990), cache.read(8990, 1)[0]
    busy = torch.randn(6000, 6000, device="cuda")
    for p in (cache.k_codes, cache.v_codes):
        p[:, 8990] = 0
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        busy = busy @ busy
        busy /= busy.abs().max()
    cache.append(k, v, 8990, stream=s)
    out = cache.attend(q, 8990, stream=s)
    got = cache.read(8990, 1, stream=s)[0]
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(got, row)
