"""The paged KV cache's operators where they can go wrong."""
import math

import pytest
import torch

import paged_ref as ref
from paged_launch import launches

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [(F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)]


@pytest.fixture(scope="module")
def pm():
    import persistent_monokernel_gb300 as pm
    pm.lib()
    torch.cuda.set_device(0)
    return pm


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- large scores

def planted(lens, places, cache, dtype, sign, hd, factor=1.0):
    """One query head per KV head, and K = sign q at the places (of those, the ones that a row has), which therefore have
    the largest scores by far: hd or so, against 6 sqrt(hd) at most."""
    q, k, v, tables, ln = ref.case(lens, 2, 2, hd, 32, cache, dtype, seed=hd)
    q = (q.to(cache) * factor).to(dtype)                  # (values that the cache's type has)
    k.mul_(factor)
    at = [[p for p in places if p < n] for n in lens]
    for i, ps in enumerate(at):
        for p in ps:
            k[int(tables[i, p // 32]), :, p % 32] = (sign * q[i]).to(cache)
    return q, k, v, tables, ln, at


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("scale", [1e3, 1e6, 1e7, 1.3e8, 1e10, 1e20])
@pytest.mark.parametrize("lens,places", [([700, 31, 1, 0, 17], [0, 3]), ([700, 300, 64], [0, 17, 40, 41, 255, 640]), ([13001], [12]),
                                         ([13001], [7, 16, 5000, 5001, 12999])])
def test_scores_far_beyond_their_steps(pm, lens, places, scale, sign, cache, dtype):
    """The largest score has all the weight, equal ones share it.  Scores of 1e5 to 1e22 are steps of up to 1e15 apart; equal rows
    of K have equal scores to the bit, all others' weight is 0, so that only the mean of the rows of V (m of them, added
    up and divided in 32 bits) and the output's half step are left."""
    for hd in (64, 128):
        q, k, v, tables, ln, at = planted(lens, places, cache, dtype, sign, hd)
        got = pm.PagedKVCache.wrap(k, v).attend(q, tables, ln, scale=sign * scale)
        for i, ps in enumerate(at):
            if not ps:
                assert not got[i].any()
                continue
            rows = torch.stack([v[int(tables[i, p // 32]), :, p % 32] for p in ps]).double()
            want, size = rows.mean(0), rows.abs().mean(0)
            bound = ref.HALF_STEP[dtype] * want.abs() + (len(ps) + 4) * 2.0 ** -23 * size + (2.0 ** -25 if dtype == F16 else 0)
            ref.check(got[i], want, bound)


@pytest.mark.parametrize("cache,dtype", TYPES)
def test_large_queries_and_keys(pm, cache, dtype):
    """The same by values of some ten thousand each, at the usual scale."""
    q, k, v, tables, ln, at = planted([700, 64, 5], [2, 33, 690], cache, dtype, 1, 128, 2.0 ** 13)
    got = pm.PagedKVCache.wrap(k, v).attend(q, tables, ln)
    for i, ps in enumerate(at):
        rows = torch.stack([v[int(tables[i, p // 32]), :, p % 32] for p in ps]).double()
        want, size = rows.mean(0), rows.abs().mean(0)
        ref.check(got[i], want, ref.HALF_STEP[dtype] * want.abs() + (len(ps) + 4) * 2.0 ** -23 * size + (2.0 ** -25 if dtype == F16 else 0))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n", [1, 16, 100, 13000])
def test_rows_of_infinitely_low_scores_are_not_empty(pm, n, dtype):
    """Every score -inf: there is no softmax (-inf minus -inf), and zeros are for rows that see no position.  Next to finite
    scores they have no weight."""
    q, k, v, tables, lens = ref.case([n, n, 0], 2, 2, 64, 16, dtype, dtype, seed=n)
    q[:] = 1.0
    for j in range(ref.cdiv(n, 16)):
        k[int(tables[0, j]), 0, :, 5] = -math.inf
        k[int(tables[1, j]), 1, :, 5] = -math.inf
    out = pm.PagedKVCache.wrap(k, v).attend(q, tables, lens)
    assert out[0, 0].isnan().all() and out[1, 1].isnan().all() and not out[2].any()
    want, bound = ref.attend(q, k.nan_to_num(0.0, neginf=0.0), v, tables, lens)
    ref.check(out[0, 1], want[0, 1], bound[0, 1])
    ref.check(out[1, 0], want[1, 0], bound[1, 0])
    last = int(tables[0, (n - 1) // 16]), 0, (n - 1) % 16
    k[last][5] = 1.0                                      # one finite score: it has all the weight
    assert torch.equal(pm.PagedKVCache.wrap(k, v).attend(q, tables, lens)[0, 0], v[last])


# ---------------------------------------------------------------- long sums

@pytest.mark.parametrize("dtype,n", [(F16, 2 ** 14), (BF16, 2 ** 17)])
def test_a_long_row_keeps_small_addends(pm, dtype, n):
    """One warp adds n slabs: a first sum S, then by turns 1/4 and 3/4 of a step of S in 32 bits.  Rounded to nearest they
    come to half a step each, cut off to nothing.  n steps are a step of the output's type, or its half."""
    head = 2.0 ** 15                                      # S = 2^7 16 head; its step in units of P = 2^7: 16 head 2^-23
    step = 16 * head * 2.0 ** -23
    k = torch.zeros(2, 8, 128, 64, dtype=dtype, device="cuda")
    v = torch.zeros_like(k)
    v[0, :, :64] = head                                   # four warps, a slab each
    v[0, :, 64::16], v[1, :, 64::16], v[1, :, :64:16] = 0.25 * step, 0.25 * step, 0.75 * step
    positions = 64 * n
    tables = torch.ones(1, positions // 128, dtype=torch.int32, device="cuda")
    tables[0, 0] = 0
    lens = torch.zeros(256, dtype=torch.int32, device="cuda")
    lens[0] = positions
    q = torch.zeros(256, 8, 64, dtype=dtype, device="cuda")
    out = pm.PagedKVCache.wrap(k, v).attend(q, tables.expand(256, -1), lens)
    want = (64 * head + 4 * step * (0.25 + (n - 2) / 2)) / positions
    low = 64 * head / positions
    assert torch.tensor(want, dtype=dtype) > torch.tensor(low, dtype=dtype)
    assert torch.equal(out[0], torch.full_like(out[0], want)) and not out[1:].any()


@pytest.mark.parametrize("cache,dtype", TYPES)
def test_weights_that_cancel(pm, cache, dtype):
    """Two positions whose scores differ by d, V = 1 and -e^d (rounded): their weights cancel up to that rounding, which shows the
    weights' own error.  Exponents below 8 round to 2^-22, exp2 adds 2^-22 and the terms of P 2^-24: 2^-21 in each weight, and
    the larger one's share, 0.67, of both in the output."""
    d = (0.2 + torch.arange(256, dtype=torch.float64) / 512).to(cache).double()
    far = torch.exp(d).to(cache).double()
    k, v = (torch.zeros(256, 1, 16, 64, dtype=cache, device="cuda") for _ in range(2))
    k[:, 0, 1, 0] = -d.cuda()
    v[:, 0, 0], v[:, 0, 1] = 1.0, -far.cuda()[:, None]
    q = torch.zeros(256, 1, 64, dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    tables, lens = torch.arange(256, dtype=torch.int32, device="cuda")[:, None], torch.full((256,), 2, dtype=torch.int32, device="cuda")
    got = pm.PagedKVCache.wrap(k, v).attend(q, tables, lens, scale=1.0)
    want = ((1 - far * torch.exp(-d)) / (1 + torch.exp(-d))).cuda()[:, None, None].expand_as(got)
    ref.check(got, want, ref.HALF_STEP[dtype] * want.abs() + 2.0 ** -20)


# ---------------------------------------------------------------- every position once

def marked(lens, group, hkv, hd, page, cache, dtype):
    """Queries of zeros (equal weights), and V that marks positions: dim d of KV head 0 those whose slab of 16 is d modulo
    hd, of head 1 those that are d modulo hd, of head 2 those whose stretch of 64 slabs is; then the same again."""
    q, k, v, tables, ln = ref.case(lens, group * hkv, hkv, hd, page, cache, dtype, seed=1)
    v.zero_()
    for i, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        ids = tables[i].long()[j // page]
        for h in range(hkv):
            v[ids, h, j % page, (j // (16, 1, 1024)[h % 3]) % hd] = 1.0
    return torch.zeros_like(q), k, v, tables, ln


def shares(n, group, hkv, hd, window=0, left_out=()):
    """[heads, hd]: what share of a row's positions each dim marks; left_out: slabs that do not count."""
    j = torch.arange(max(0, n - window) if window else 0, n)
    for s in left_out:
        j = j[j // 16 != s]
    return torch.stack([torch.bincount((j // d) % hd, minlength=hd) for d in (16, 1, 1024)]).double()[[h % 3 for h in range(hkv)]] \
        .repeat_interleave(group, 0) / max(len(j), 1)


def mark_bound(want, dtype):
    """Weights are a power of two, so that all sums are exact: 1 / n and the product with it round, and the output."""
    return (ref.HALF_STEP[dtype] + 2.0 ** -22) * want + (2.0 ** -25 if dtype == F16 else 0)


def check_marks(pm, c, group, lens, window):
    q, k, v, tables, ln = c
    got = pm.PagedKVCache.wrap(k, v).attend(q, tables, ln, window=window)
    want = torch.stack([shares(n, group, k.shape[1], k.shape[3], window) for n in lens]).cuda()
    ref.check(got, want, mark_bound(want, q.dtype))


MARKED = [[40000], [30000, 29999], [13001, 0, 5], [5000], [4097, 1024], [1023] * 5, [300] * 40, [8000] * 4, list(range(1, 2400, 37)),
          [20000] + [17] * 90, [33000] + [40] * 39]


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("lens", MARKED, ids=lambda x: f"{len(x)}x{max(x)}")
def test_every_position_counts_once(pm, lens, cache, dtype):
    """A slab (or a position, or a part) left out or counted twice shows, whatever the row's length."""
    for hd in (64, 128):
        c = marked(lens, 2, 3, hd, 64, cache, dtype)
        for window in (0, max(lens) - 3, 1000):
            check_marks(pm, c, 2, lens, window)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_marks_tell_of_one_slab(dtype):
    """What the two tests around this one would see if a kernel left one slab out: more than they let pass."""
    for n in (40000, 66000):
        want = shares(n, 1, 3, 64)
        for s in (0, 7, n // 32, n // 16 - 1):
            assert bool(((shares(n, 1, 3, 64, 0, [s]) - want).abs() > 2 * mark_bound(want, dtype)).any())


# lengths, heads per KV head, KV heads, head_dim, page; the launch (clusters, warps, parts, long rows first)
REACHED = [([66000, 40, 0, 1500] + [100] * 36, 2, 4, 64, 128, (8, 4, 1, 1)), ([33000, 40, 0, 1500] + [100] * 36, 1, 4, 128, 128, (8, 4, 1, 1)),
           ([0] * 255 + [6000], 2, 2, 128, 64, (2, 4, 1, 1)), ([4200] + [33, 0] * 127 + [16], 1, 2, 128, 64, (1, 4, 1, 1)),
           ([12000, 0, 900, 15] * 50, 9, 2, 128, 64, (4, 4, 1, 1)), ([2100, 7, 0, 700] * 40, 1, 3, 128, 64, (1, 4, 1, 1)),
           ([4100] + [50, 0, 1, 300] * 64, 4, 2, 128, 64, (2, 4, 1, 0)), ([9000] + [80] * 298 + [0], 2, 2, 128, 64, (4, 4, 1, 0)),
           ([40000] + [20] * 279, 3, 1, 128, 256, (8, 4, 1, 0)), ([500] * 400, 2, 2, 64, 32, (1, 4, 1, 0)), ([8000], 4, 5, 128, 64, (8, 8, 1, 0)),
           ([40000], 17, 3, 64, 64, (4, 4, 11, 0)), ([13000] * 4, 8, 1, 128, 16, (4, 4, 17, 0)), ([1000] * 24, 4, 5, 128, 64, (2, 4, 1, 0))]


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("lens,group,hkv,hd,page,launch", REACHED, ids=lambda x: f"{len(x)}x{max(x)}" if isinstance(x, list) else None)
def test_each_kind_of_launch(pm, tmp_path, lens, group, hkv, hd, page, launch, cache, dtype):
    """Rows that need all CTAs of their launch, few and none, with the launch that the rule chooses for them."""
    width = ref.cdiv(max(lens), page)
    chosen, = launches([(len(lens), group, hkv, hd, page, width, 0)], str(tmp_path),
                       torch.cuda.get_device_properties(0).multi_processor_count)
    assert chosen == launch
    c = marked(lens, group, hkv, hd, page, cache, dtype)
    for window in (0, max(lens) - 3):
        check_marks(pm, c, group, lens, window)
    # Equal weights of random values.  What rounds is the sum of V: half a step of 32 bits for each slab of a warp, a step
    # for each of a slab's two times 17 addends, which the products cut, and the joins' 40 half ones.
    q, k, v, tables, ln = ref.case(lens, group * hkv, hkv, hd, page, cache, dtype, seed=2)
    got = pm.PagedKVCache.wrap(k, v).attend(q.zero_(), tables, ln)
    for i, n in enumerate(lens):
        if not n:
            assert not got[i].any()
            continue
        j = torch.arange(n, device="cuda")
        rows = v[tables[i].long()[j // page], :, j % page].double()
        want, size = (x.mean(0).repeat_interleave(group, 0) for x in (rows, rows.abs()))
        chain = n // (16 * chosen.cl * chosen.cw * chosen.parts) + 8
        bound = (chain / 2 + 64) * 2.0 ** -23 * size
        ref.check(got[i], want, bound + ref.HALF_STEP[dtype] * (want.abs() + bound) + (2.0 ** -25 if dtype == F16 else 0))


# ---------------------------------------------------------------- what torch has to know

def test_forward_mode_derivatives_are_refused(pm):
    import torch.autograd.forward_ad as fwad
    q, k, v, tables, lens = ref.case([20, 5], 4, 2, 64, 16, F16, F16)
    cache, kv4 = pm.PagedKVCache.wrap(k, v), pm.KV4Cache(2, 64, 16)
    x = torch.zeros(3, 2, 64, dtype=F16, device="cuda")
    slots = ints([1, 2, 3])
    kv4.append(x, x, 0)
    want = cache.attend(q, tables, lens)
    with fwad.dual_level():
        dual = fwad.make_dual(q, torch.ones_like(q))
        dx = fwad.make_dual(x, torch.ones_like(x))
        pool = fwad.make_dual(k.clone(), torch.ones_like(k))
        for call in (lambda: cache.attend(dual, tables, lens), lambda: cache.append(dx, x, slots), lambda: cache.append(x, dx, slots),
                     lambda: pm.PagedKVCache.wrap(pool, v).attend(q, tables, lens), lambda: kv4.append(dx, x, 0),
                     lambda: kv4.attend(dual[:, :2], 0), lambda: cache.attend(q, tables, lens, out=fwad.make_dual(q.clone(), q)),
                     lambda: kv4.read(0, 3, out=(dx.clone(), x.clone()))):
            with pytest.raises(ValueError, match="tangent"):
                call()
        with torch.inference_mode():                      # no derivatives are asked for
            assert torch.equal(cache.attend(dual, tables, lens), want)
        assert torch.equal(cache.attend(fwad.unpack_dual(dual).primal, tables, lens), want)


def test_writes_are_seen_by_autograd(pm):
    """A tensor that a backward pass has kept and a call has written since is an error, as with any write in place."""
    k, v = (torch.zeros(2, 2, 16, 64, dtype=F16, device="cuda") for _ in range(2))
    cache = pm.PagedKVCache.wrap(k, v)
    x = torch.ones(3, 2, 64, dtype=F16, device="cuda")
    t = pm.PageTables(2, 1, 2, 16)
    lens, tables = ints([3, 0]), ints([[0], [1]])
    for kept in (k, v):
        w = torch.ones_like(kept, requires_grad=True)
        y = (kept * w).sum()
        cache.append(x, x, ints([0, 1, 2]))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()

    def bumped(call, *tensors):
        was = [a._version for a in tensors]
        call()
        return all(a._version > b for a, b in zip(tensors, was))

    q, out = torch.ones(2, 4, 64, dtype=F16, device="cuda"), torch.empty(2, 4, 64, dtype=F16, device="cuda")
    assert bumped(lambda: cache.append(x, x, ints([0, 1, 2])), k, v)
    assert bumped(lambda: cache.attend(q, tables, lens, out=out), out)
    assert not any(bumped(lambda: cache.attend(q, tables, lens), a) for a in (k, v, q, tables, lens))
    assert bumped(lambda: t.plan(ints([1, 1]), 2), t.tables, t.lens, t.free, t.n_free, t.status)
    kv4 = pm.KV4Cache(2, 64, 16)
    a, b = x.clone(), x.clone()
    assert bumped(lambda: kv4.append(x, x, 0), kv4.k_codes, kv4.k_scales, kv4.v_codes, kv4.v_scales)
    assert bumped(lambda: kv4.read(0, 3, out=(a, b)), a, b)
    assert bumped(lambda: kv4.attend(x, 0, out=a), a)
    with torch.inference_mode():                          # tensors without a version
        free = [torch.zeros_like(k) for _ in range(2)]
        o = torch.empty_like(q)
    pm.PagedKVCache.wrap(*free).append(x, x, ints([0, 1, 2]))
    pm.PagedKVCache.wrap(*free).attend(q, tables, lens, out=o)
    assert torch.equal(o, out)


def test_sync_of_another_stream(pm):
    """A plan on a stream of its own: sync on that stream waits for it."""
    t = pm.PageTables(2, 4, 6, 16)
    s = torch.cuda.Stream()
    new = ints([100, 0])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    t.plan(new, 200, stream=s)
    assert t.sync(stream=s) == 3
    assert t.sync() == 0 and t.sync(stream=s) == 0
    with pytest.raises(ValueError, match="stream"):
        class Elsewhere:
            device = torch.device("cuda", 99)
        t.sync(stream=Elsewhere())


def test_caches_that_cannot_be_are_refused_at_once(pm):
    for args in ((4, 2, 64, 8), (4, 2, 96), (0, 2, 64), (4, 0, 64), (4, 1025, 64), (2 ** 27, 1, 64), (4, 2, 64, 24), (4, 2, 64, 0),
                 (4, 2, 64, 2 ** 31)):
        was = torch.cuda.memory_allocated(), torch.cuda.max_memory_allocated()
        with pytest.raises((pm.LFError, ValueError)):
            pm.PagedKVCache(*args)
        assert (torch.cuda.memory_allocated(), torch.cuda.max_memory_allocated()) == was
    with pytest.raises(ValueError):
        pm.PagedKVCache(4, 2, 64, dtype=F32)
    k, v = (torch.zeros(4, 2, 24, 64, dtype=F16, device="cuda") for _ in range(2))
    for bad in ((k, v), (k[:, :, :16, :32], v[:, :, :16, :32]), (k[:, :, :16], k[:, :, :16])):
        with pytest.raises(pm.LFError):
            pm.PagedKVCache.wrap(*bad)
