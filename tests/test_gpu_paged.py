"""The paged KV cache's operators on the GPU, against their definitions in lists and 64 bits (paged_ref.py)."""
import random

import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def pm():
    import persistent_monokernel_gb300 as pm
    pm.lib()
    torch.cuda.set_device(0)
    return pm


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- attend

def attend(pm, c, **kw):
    q, k, v, tables, lens = c
    got = pm.PagedKVCache.wrap(k, v).attend(q, tables, lens, **kw)
    assert got.dtype == q.dtype and got.shape == q.shape
    ref.check(got, *ref.attend(q, k, v, tables, lens, kw.get("window", 0), kw.get("scale", 0.0)))
    return got


TYPES = [(F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)]
GROUPS = [(20, 5, 128), (16, 4, 64), (4, 4, 64), (8, 1, 128), (9, 1, 64), (32, 2, 128), (40, 1, 64), (17, 1, 128)]


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("heads,hkv,hd", GROUPS)
def test_groups_and_types(pm, heads, hkv, hd, cache, dtype):
    attend(pm, ref.case([77, 0, 1, 200], heads, hkv, hd, 32, cache, dtype, seed=heads))


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("by_head", [True, False])
def test_lengths(pm, page, by_head):
    """One to several pages, at and around the ends of slabs and pages; what lies behind a row's end is NaN."""
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 255, 256, 257, 511, 513, 1000]
    for dtype in (F16, F32):
        attend(pm, ref.case(lens, 8, 2, 128, page, F16, dtype, seed=page, by_head=by_head))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 1000, 5000])
def test_windows(pm, hd, window):
    attend(pm, ref.case([0, 1, 16, 99, 100, 101, 1023, 3000], 4, 2, hd, 48, BF16, BF16, seed=window), window=window)


# what decides the launch: few rows of many positions (parts, and CTAs of eight warps), and many rows
SHAPES = [((1, 5), [12288 + 7]), ((1, 2), [4096 + 33]), ((1, 2), [2048]), ((1, 1), [40000]), ((2, 4), [13000, 14000, 0]),
          ((2, 8), [300] * 40), ((1, 2), list(range(0, 1200, 3))), ((1, 1), [16 * i for i in range(60)])]


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("heads,lens", SHAPES)
def test_launches(pm, heads, lens, cache, dtype):
    group, hkv = heads
    c = ref.case(lens, 3 * group * hkv, hkv, 64, 64, cache, dtype, seed=len(lens))
    a = attend(pm, c)
    assert torch.equal(a, attend(pm, c))                  # equal calls, equal bits


def test_parts_with_windows_and_short_rows(pm):
    """A wide table where one row needs all parts, one few and one none, with and without a window."""
    c = ref.case([30000, 5, 700, 0], 8, 2, 128, 64, F16, F16, seed=3)
    for window in (0, 14000, 20, 29999):
        attend(pm, c, window=window)


LONG_FIRST = [(4, 128, [2100, 0, 5, 16, 17, 700, 700, 1999] * 10), (2, 64, [4100] + [i % 40 for i in range(199)]),
              (4, 128, [0] * 30 + [4200, 1] + [33] * 18), (1, 64, [0] * 255 + [5000])]


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("hkv,hd,lens", LONG_FIRST)
def test_long_rows_first(pm, hkv, hd, lens, cache, dtype):
    """More rows than run at a time, of few or many lengths, equal ones and none among them: each is taken once."""
    attend(pm, ref.case(lens, hkv * (9 if hkv == 2 else 2), hkv, hd, 64, cache, dtype, seed=hkv))


@pytest.mark.parametrize("lens", [[33000, 40, 0, 1500] + [100] * 36])
def test_clusters_of_eight_in_rounds(pm, lens):
    attend(pm, ref.case(lens, 8, 4, 64, 128, F16, F16, seed=8))
    attend(pm, ref.case(lens, 8, 4, 64, 128, F16, F16, seed=8), window=20000)


@pytest.mark.parametrize("lens", [[40, 33], [13000, 12999]])
def test_tables_narrower_than_the_lengths_and_wider(pm, lens):
    q, k, v, tables, ln = ref.case(lens, 4, 2, 64, 16, F16, F16, width=900)
    for width in (1, 2, 3, 800, 900):
        for window in (0, 30):
            attend(pm, (q, k, v, tables[:, :width], ln), window=window)
    out = pm.PagedKVCache.wrap(k, v).attend(q, tables[:, :0], ln)
    assert torch.equal(out, torch.zeros_like(q))


@pytest.mark.parametrize("lens", [[300, 120, 64], [20000]])
def test_pages_that_the_pool_does_not_have_are_left_out(pm, lens):
    q, k, v, tables, ln = ref.case(lens, 8, 2, 128, 16, BF16, BF16)
    rng = random.Random(5)
    for i in range(len(lens)):
        for _ in range(ref.cdiv(lens[i], 16) // 3):
            tables[i, rng.randrange(ref.cdiv(lens[i], 16))] = rng.choice([-1, -2 ** 31, len(k), 2 ** 31 - 1])
    attend(pm, (q, k, v, tables, ln))
    attend(pm, (q, k, v, tables, ln), window=50)
    tables[0] = -1
    out = attend(pm, (q, k, v, tables, ln))
    assert not out[0].any()


def test_lengths_that_are_none(pm):
    q, k, v, tables, _ = ref.case([40, 40, 40], 4, 2, 64, 16, F16, F16)
    lens = ints([-1, -2 ** 31, 2 ** 31 - 1])
    attend(pm, (q, k, v, tables[:, :2], lens))            # the last row: all that the table has
    attend(pm, (q, k, v, tables[:, :2], lens), window=2 ** 31 - 1)


def test_one_table_for_all_rows_and_pages_twice(pm):
    q, k, v, tables, _ = ref.case([100, 1, 1], 4, 2, 64, 16, F16, F16)
    attend(pm, (q, k, v, tables[:1].expand(3, -1), ints([100, 50, 3])))
    tables[0, 2] = tables[0, 0]
    attend(pm, (q, k, v, tables, ints([100, 1, 1])))


@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 4.0])
def test_scales(pm, cache, dtype, scale):
    """Scores from small to far apart (one position then has all the weight)."""
    attend(pm, ref.case([500, 31], 8, 2, 128, 64, cache, dtype, seed=9), scale=scale)


def test_scores_that_grow_along_the_row(pm):
    """The running reference has to move many times, and far."""
    for dtype in (F16, F32):
        q, k, v, tables, lens = ref.case([1500], 4, 1, 64, 16, F16, dtype, seed=2)
        q[:] = 1.0
        for j in range(94):
            k[int(tables[0, j])] = torch.linspace(0.2 * j, 0.2 * (j + 1), 16, device="cuda").half()[None, :, None].expand(1, 16, 64)
        attend(pm, (q, k, v, tables, lens))


def test_small_and_large_fp32_queries(pm):
    for factor in (1e-30, 1e-4, 1.0, 1e4):
        q, *rest = ref.case([200, 17], 8, 2, 64, 16, F16, F32, seed=4)
        attend(pm, (q * factor, *rest), scale=0.125 / factor if factor < 1 else 0.125 / factor)


def test_infinite_and_nan_positions_spoil_only_rows_that_see_them(pm):
    q, k, v, tables, lens = ref.case([64, 64, 64], 4, 2, 64, 16, F16, F16, seed=6)
    k[int(tables[0, 1]), 0, 3] = float("nan")
    v[int(tables[1, 1]), 1, 3] = float("inf")
    got = pm.PagedKVCache.wrap(k, v).attend(q, tables, lens)
    assert got[0, :2].isnan().all() and got[0, 2:].isfinite().all()
    assert got[1, :2].isfinite().all() and not got[1, 2:].isfinite().any()
    want, bound = ref.attend(q, k, v, tables, lens)
    ref.check(got[2], want[2], bound[2])
    attend(pm, (q, k, v, tables, ints([16, 16, 64])))     # those positions are no longer seen


def test_strided_queries_and_outputs(pm):
    q, k, v, tables, lens = ref.case([77, 20, 130], 8, 2, 128, 32, F16, F16)
    want, bound = ref.attend(q, k, v, tables, lens)
    cache = pm.PagedKVCache.wrap(k, v)
    wide = torch.full((3, 14, 160), 9.0, dtype=F16, device="cuda")
    wide[:, 3:11, :128] = q
    out = torch.full((8, 5, 128), 7.0, dtype=F16, device="cuda")
    got = cache.attend(wide[:, 3:11, :128], tables, lens, out=out.transpose(0, 1)[1:4])
    assert got.data_ptr() == out[:, 1:].data_ptr()
    ref.check(got, want, bound)
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 4] == 7).all())   # other rows are left as they were
    same = q[:1].expand(3, -1, -1)                        # one query for all rows
    ref.check(cache.attend(same, tables, lens), *ref.attend(same, k, v, tables, lens))


def test_no_sequences(pm):
    _, k, v, tables, lens = ref.case([5], 4, 2, 64, 16, F16, F16)
    assert pm.PagedKVCache.wrap(k, v).attend(torch.empty(0, 4, 64, dtype=F16, device="cuda"), tables[:0], lens[:0]).shape == (0, 4, 64)


def test_slices_of_one_pool_for_k_and_v(pm):
    q, k, v, tables, lens = ref.case([77, 20], 4, 2, 64, 16, F16, F16)
    both = torch.stack((k, v), 1)
    attend(pm, (q, both[:, 0], both[:, 1], tables, lens))


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("cache,dtype", TYPES)
@pytest.mark.parametrize("hd,page,by_head", [(128, 16, True), (64, 48, False), (128, 64, False)])
def test_append(pm, cache, dtype, hd, page, by_head):
    n_pages, hkv, n = 7, 3, 61
    k, v, g = ref.pools(n_pages, hkv, page, hd, cache, 3, by_head, fill=5.0)
    rows = torch.randn(n, 4 * hkv * hd, generator=g, device="cuda").to(dtype)
    x, y = (rows[:, i * hkv * hd:(i + 1) * hkv * hd].unflatten(1, (hkv, hd)) for i in (1, 3))
    slots = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(1))[:n].tolist()
    for i, s in zip((0, 7, 8, 60), (-1, n_pages * page, -2 ** 31, 2 ** 31 - 1)):
        slots[i] = s
    want = [k.clone(), v.clone()]
    for t, s in enumerate(slots):
        if 0 <= s < n_pages * page:
            for w, r in zip(want, (x, y)):
                w[s // page, :, s % page] = r[t].to(cache)
    cache_ = pm.PagedKVCache.wrap(k, v)
    cache_.append(x, y, ints(slots))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    cache_.append(x[:0], y[:0], ints([]))
    assert torch.equal(k, want[0])


def test_append_rounds_like_a_conversion(pm):
    """Halfway cases, overflow, subnormals, infinities and NaN of FP32 rows, and 16-bit rows bit by bit."""
    x = torch.tensor([0.0, -0.0, 1 + 2.0 ** -11, 1 + 3 * 2.0 ** -11, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 65504, 65519.9, 65520, 1e38, 3.4e38,
                      -1e30, 2.0 ** -24, 2.0 ** -25, 3 * 2.0 ** -26, 1e-40, float("inf"), -float("inf"), float("nan"), 2.0 ** -133],
                     device="cuda").repeat(4)[:64].view(1, 1, 64)
    for dt in (F16, BF16):
        k, v, _ = ref.pools(1, 1, 16, 64, dt, 0)
        pm.PagedKVCache.wrap(k, v).append(x, -x, ints([5]))
        for got, want in ((k[0, 0, 5], x.to(dt)), (v[0, 0, 5], (-x).to(dt))):
            want = want.view(-1)
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
            assert torch.equal(got[~want.isnan()].view(torch.int16), want[~want.isnan()].view(torch.int16))
        bits = torch.arange(-2 ** 15, 2 ** 15, device="cuda").to(torch.int16).view(1024, 1, 64)
        k, v, _ = ref.pools(64, 1, 16, 64, dt, 0)
        pm.PagedKVCache.wrap(k, v).append(bits.view(dt), bits.view(dt), torch.arange(1024, dtype=torch.int32, device="cuda"))
        assert torch.equal(k.view(-1, 64).view(torch.int16), bits.view(-1, 64))


def test_pages_far_apart(pm):
    """Byte offsets beyond 32 bits, within the pool and the rows: pages 3 GB apart."""
    apart = 3 * 2 ** 29
    store = torch.zeros(2 * apart + 2 * 2 * 16 * 64, dtype=F16, device="cuda")
    k, v = (store[o:].as_strided((3, 2, 16, 64), (apart, 1024, 64, 1)) for o in (0, 2048))
    g = torch.Generator("cuda").manual_seed(1)
    x, y = (torch.randn(48, 2, 64, generator=g, device="cuda").half() for _ in range(2))
    slots = torch.randperm(48, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    cache = pm.PagedKVCache.wrap(k, v)
    cache.append(x, y, slots)
    for pool, r in ((k, x), (v, y)):
        assert torch.equal(torch.cat([pool[p].transpose(0, 1) for p in range(3)])[slots.long()], r)
    q = torch.randn(1, 4, 64, generator=g, device="cuda").half()
    attend(pm, (q, k, v, ints([[2, 0, 1]]), ints([48])))


# ---------------------------------------------------------------- plan

def same(t, b, got=None, want=None):
    assert t.lens.tolist() == b.lens
    n_free = int(t.n_free)
    assert t.free[:n_free].tolist() == b.free
    for i, row in enumerate(t.tables.tolist()):
        used = ref.cdiv(b.lens[i], b.page)
        assert row[:used] == b.tables[i][:used]
    if got is not None:
        assert [x.tolist() for x in got] == list(want[:3])


@pytest.mark.parametrize("n,max_pages,n_pages,page", [(1, 4, 4, 16), (5, 9, 20, 16), (33, 6, 120, 48), (300, 40, 4000, 64), (2000, 3, 5000, 32)])
def test_plans_of_many_steps(pm, n, max_pages, n_pages, page):
    """Random growth, drafts taken back, rows ended and begun anew; steps that do not fit change nothing."""
    rng = random.Random(n)
    t, b = pm.PageTables(n, max_pages, n_pages, page), ref.Batch(n, max_pages, n_pages, page)
    same(t, b)
    failed = 0
    for step in range(30):
        room = max(1, n_pages * page // (2 * n))
        n_new = [rng.choice([0, 1, 1, rng.randrange(room)]) for _ in range(n)]
        keep = None if step % 3 == 0 else [rng.choice([0, max(0, x - rng.randrange(5)), x, 10 ** 9]) for x in b.lens]
        most = rng.choice([sum(n_new), sum(n_new) + rng.randrange(70), 5000 + sum(n_new), max(0, sum(n_new) - 1)])
        want = b.plan(n_new, most, keep)
        got = t.plan(ints(n_new), most, None if keep is None else ints(keep))
        same(t, b, got, want)
        assert t.sync() == (3 if want[3] else 0)
        failed += want[3]
        if step == 20:
            n_new, keep = [0] * n, [0] * n
            same(t, b, t.plan(ints(n_new), 8, ints(keep)), b.plan(n_new, 8, keep))
            assert int(t.n_free) == n_pages
    assert failed


def test_a_plan_taken_back_finds_the_same_pages(pm):
    t = pm.PageTables(6, 50, 200, 16)
    t.plan(ints([40, 0, 100, 7, 16, 33]), 256)
    base = t.lens.clone()
    first = t.plan(ints([5, 30, 0, 100, 1, 16]), 300)
    state = [x.clone() for x in (t.tables, t.lens, t.free, t.n_free)]
    for _ in range(3):
        again = t.plan(ints([5, 30, 0, 100, 1, 16]), 300, keep=base)
        assert all(torch.equal(a, b) for a, b in zip(again, first))
        assert all(torch.equal(a, b) for a, b in zip((t.tables, t.lens, t.free, t.n_free), state))


@pytest.mark.parametrize("most", [0, 1, 3, 4, 5, 4095, 4096, 4097, 9999])
def test_most_tokens(pm, most):
    """Entries up to max_tokens are written, and none behind them."""
    t, b = pm.PageTables(3, 700, 900, 16), ref.Batch(3, 700, 900, 16)
    new = [most // 3, 0, most - most // 3]
    same(t, b, t.plan(ints(new), most), b.plan(new, most))
    assert t.sync() == 0


def test_plans_that_fail(pm):
    """Every kind of failure leaves the state as it was, and the first one is told of."""
    t, b = pm.PageTables(2, 4, 6, 16), ref.Batch(2, 4, 6, 16)
    same(t, b, t.plan(ints([20, 30]), 50), b.plan([20, 30], 50))
    bad = [([100, 0], 200, None, 3), ([0, 36], 60, None, 3), ([44, 34], 90, None, 3), ([3, 3], 5, None, 3),
           ([-1, 2], 60, None, 1), ([1, 1], 60, [-1, 5], 1), ([2 ** 31 - 1, 2 ** 31 - 1], 60, None, 3)]
    for n_new, most, keep, status in bad:
        for m in (most, most + 5000):
            if status == 3 and sum(n_new) <= m and n_new == [3, 3]:
                continue
            got = t.plan(ints(n_new), m, None if keep is None else ints(keep))
            assert [x.tolist() for x in got] == [[-1] * m, [0] * m, [0] * 3]
            same(t, b)
            assert t.sync() == status and t.sync() == 0
    t.plan(ints([100, 0]), 200), t.plan(ints([-1, 0]), 200)
    assert t.sync() == 3
    for field, value in (("lens", [20, 65]), ("lens", [-1, 30]), ("n_free", [7]), ("n_free", [-1])):
        x = getattr(t, field)
        was = x.clone()
        x.copy_(ints(value))
        assert (t.plan(ints([1, 1]), 8)[0] == -1).all() and t.sync() == 1
        assert x.tolist() == value
        x.copy_(was)
    t.n_free.fill_(3)                                      # more pages given back than the pool has places for
    assert (t.plan(ints([0, 0]), 8, keep=ints([0, 0]))[0] == -1).all() and t.sync() == 1
    t.n_free.fill_(2)
    same(t, b, t.plan(ints([1, 1]), 8), b.plan([1, 1], 8))


def test_no_rows(pm):
    t = pm.PageTables(0, 4, 6, 16)
    slots, positions, offsets = t.plan(ints([]), 10)
    assert slots.tolist() == [-1] * 10 and positions.tolist() == [0] * 10 and offsets.tolist() == [0]
    assert t.sync() == 0 and int(t.n_free) == 6


def test_the_most_rows(pm):
    n = 8192
    t, b = pm.PageTables(n, 2, 2 * n, 16), ref.Batch(n, 2, 2 * n, 16)
    for new, keep in (([i % 23 for i in range(n)], None), ([1] * n, [i % 19 for i in range(n)])):
        same(t, b, t.plan(ints(new), sum(new), keep and ints(keep)), b.plan(new, sum(new), keep))
    with pytest.raises(pm.LFError):
        pm.PageTables(n + 1, 2, 6, 16).plan(ints([0] * (n + 1)), 1)


def test_tables_as_a_slice_of_wider_ones(pm):
    wide = torch.full((3, 12), 77, dtype=torch.int32, device="cuda")
    t = pm.PageTables.wrap(wide[:, 2:8], ints([0, 0, 0]), ints([3, 1, 4, 0, 5, 2]), ints([6]), 16)
    t.plan(ints([20, 1, 40]), 61)
    assert t.tables[0, :2].tolist() == [2, 5] and t.tables[1, :1].tolist() == [0] and t.tables[2, :3].tolist() == [4, 1, 3]
    assert bool((wide[:, :2] == 77).all()) and bool((wide[:, 8:] == 77).all()) and int(t.n_free) == 0


# ---------------------------------------------------------------- together

class Dense:
    """The batch as plain tensors: every row's K and V, one behind the other."""

    def __init__(self, n, hkv, hd, dtype):
        self.rows = [[torch.empty(0, hkv, hd, dtype=dtype, device="cuda") for _ in range(2)] for _ in range(n)]

    def step(self, k, v, offsets, n_new, keep=None):
        for i, r in enumerate(self.rows):
            for j, x in ((0, k), (1, v)):
                r[j] = torch.cat((r[j][:None if keep is None else keep[i]], x[offsets[i]:offsets[i] + n_new[i]].to(r[j].dtype)))

    def attend(self, q):
        n, heads, hd = q.shape
        lens = [len(r[0]) for r in self.rows]
        k, v = (torch.zeros(n, x.shape[1], max(max(lens), 16), hd, dtype=x.dtype, device="cuda") for x in self.rows[0])
        for i, r in enumerate(self.rows):
            k[i, :, :lens[i]], v[i, :, :lens[i]] = r[0].transpose(0, 1), r[1].transpose(0, 1)
        return ref.attend(q, k, v, torch.arange(n, dtype=torch.int32, device="cuda")[:, None], lens)


@pytest.mark.parametrize("cache_t,dtype,hd", [(F16, F16, 128), (BF16, F32, 64)])
def test_a_batch_served(pm, cache_t, dtype, hd):
    """Prompts, decode steps, drafts taken back, rows that end and begin anew: plan, append and attend as a program runs
    them, two layers on one plan."""
    n, hkv, heads, page, most = 6, 2, 8, 16, 128
    t = pm.PageTables(n, 20, 60, page)
    layers = [pm.PagedKVCache(60, hkv, hd, page, cache_t) for _ in range(2)]
    dense = [Dense(n, hkv, hd, cache_t) for _ in layers]
    g = torch.Generator("cuda").manual_seed(4)
    steps = [([10, 0, 33, 16, 1, 40], None), ([1] * 6, None), ([4, 4, 0, 4, 4, 4], None), ([1] * 6, [9, 1, 34, 19, 3, 44]),
             ([0, 30, 1, 1, 1, 1], [0, 0, 34, 5, 3, 44]), ([1] * 6, None), ([1, 0, 1, 1, 0, 1], None)]
    for n_new, keep in steps:
        lens = t.lens.tolist()
        slots, positions, offsets = t.plan(ints(n_new), most, keep and ints(keep))
        kept = [min(a, b) for a, b in zip(lens, keep or lens)]
        assert positions[:sum(n_new)].tolist() == [p for a, m in zip(kept, n_new) for p in range(a, a + m)]
        for cache, d in zip(layers, dense):
            qkv = torch.randn(most, (heads + 2 * hkv) * hd, generator=g, device="cuda").to(dtype).unflatten(1, (-1, hd))
            _, k, v = qkv.split((heads, hkv, hkv), 1)
            cache.append(k, v, slots)                      # the rows of padding go nowhere
            d.step(k, v, offsets.tolist(), n_new, kept)
            q = torch.randn(n, heads, hd, generator=g, device="cuda").to(dtype)
            ref.check(cache.attend(q, t.tables, t.lens), *d.attend(q))
    assert t.sync() == 0


@pytest.mark.parametrize("lens", [[100, 3, 0, 260], [12400, 13000]])
def test_captured_steps(pm, lens):
    """A decode step captured once and replayed with other inputs, in two graphs that share the pools: as the same
    steps run eagerly."""
    n, hkv, heads, hd, page, steps = len(lens), 2, 8, 64, 16, 5
    width = ref.cdiv(max(lens) + 2 * steps, page)
    n_pages = sum(ref.cdiv(x + 2 * steps, page) for x in lens)
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    inputs = torch.randn(2 * steps, n, heads + 2 * hkv, hd, generator=g, device="cuda").half()

    def make():
        t, c = pm.PageTables(n, width, n_pages, page), pm.PagedKVCache(n_pages, hkv, hd, page)
        slots, *_ = t.plan(ints(lens), sum(lens))
        gg = torch.Generator("cuda").manual_seed(2)
        c.append(*(torch.randn(sum(lens), hkv, hd, generator=gg, device="cuda").half() for _ in range(2)), slots)
        return t, c

    def step(t, c, x):
        slots, *_ = t.plan(one, n)
        q, k, v = x.split((heads, hkv, hkv), 1)
        c.append(k, v, slots)
        return c.attend(q, t.tables, t.lens)

    t, c = make()
    want = [step(t, c, x).clone() for x in inputs]
    final = t.lens.tolist(), c.k.clone()
    t, c = make()
    x = inputs[0].clone()
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(t, c, x)
        graphs.append((graph, out))
    for i, y in enumerate(inputs):
        x.copy_(y)
        graph, out = graphs[i % 2]
        graph.replay()
        assert torch.equal(out, want[i]), i
    assert (t.lens.tolist()) == final[0] and torch.equal(c.k, final[1])


def test_calls_on_other_streams(pm):
    """Two caches at once, each on a stream of its own, with temporaries that are let go of at once."""
    cases = [ref.case([13000], 8, 2, 64, 16, F16, F16, seed=1), ref.case([500] * 20, 8, 2, 64, 16, F16, F16, seed=2)]
    caches = [pm.PagedKVCache.wrap(c[1], c[2]) for c in cases]
    want = [c.attend(*x[:1], *x[3:]) for c, x in zip(caches, cases)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, x, s in zip(caches, cases, streams):
            q, tables, lens = x[0].clone(), x[3].clone(), x[4].clone()
            s.wait_stream(torch.cuda.current_stream())
            torch.cuda._sleep(1000000)
            got.append(c.attend(q, tables, lens, stream=s))
            del q, tables, lens
            [torch.full((8,), 1 << 20, dtype=torch.int32, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])
    t = pm.PageTables(2, 4, 8, 16)
    slots, _, offsets = t.plan(ints([5, 20]), 25, stream=streams[0])
    streams[0].synchronize()
    assert slots[:6].tolist() == [0, 1, 2, 3, 4, 16] and offsets.tolist() == [0, 5, 25]


def test_refusals_of_the_binding(pm):
    q, k, v, tables, lens = ref.case([20, 5], 4, 2, 64, 16, F16, F16)
    cache = pm.PagedKVCache.wrap(k, v)
    out = cache.attend(q, tables, lens)
    for bad in ((q.double(), tables, lens), (q[..., ::2], tables, lens), (q[0], tables, lens), (q, tables.long(), lens), (q, tables[0], lens),
                (q, tables[:1], lens), (q, tables.t().contiguous().t(), lens), (q, tables, lens.long()), (q, tables, lens[:1]),
                (q, tables, lens.cpu()), (q.cpu(), tables, lens), (q, tables.cpu(), lens), (q, None, lens),
                (q.float().requires_grad_(), tables, lens)):
        with pytest.raises(ValueError):
            cache.attend(*bad)
    for bad in (dict(window=2 ** 31), dict(scale=1e-300), dict(out=q[:1]), dict(out=out.cpu())):
        with pytest.raises(ValueError):
            cache.attend(q, tables, lens, **bad)
    for bad in (dict(window=-1), dict(scale=float("nan")), dict(out=q), dict(out=out.float())):
        with pytest.raises(pm.LFError):
            cache.attend(q, tables, lens, **bad)
    with pytest.raises(pm.LFError):
        cache.attend(q.bfloat16(), tables, lens)
    with pytest.raises(pm.LFError):
        cache.attend(q[:, :3], tables, lens)              # no multiple of the KV heads
    x = torch.zeros(3, 2, 64, dtype=F16, device="cuda")
    for bad in ((x[:, :1], x, ints([1, 2, 3])), (x, x[:2], ints([1, 2, 3])), (x, x, ints([1, 2])), (x, x, ints([1, 2, 3]).long()),
                (x, x, torch.zeros(6, dtype=torch.int32, device="cuda")[::2]), (x.float().requires_grad_(), x.float(), ints([1, 2, 3]))):
        with pytest.raises(ValueError):
            cache.append(*bad)
    for bad in ((x.bfloat16(), x.bfloat16()), (x.float(), x)):
        with pytest.raises(pm.LFError):
            cache.append(*bad, ints([1, 2, 3]))
    for bad in ((k, v.bfloat16()), (k, v[:1]), (k.float(), v.float()), (k[..., :32], v[..., ::2]), (k, torch.stack((v, v), 1)[:, 0]), (k[0], v[0])):
        with pytest.raises(ValueError):
            pm.PagedKVCache.wrap(*bad)
    with pytest.raises(pm.LFError):
        pm.PagedKVCache(4, 2, 64, page=8).append(x, x, ints([1, 2, 3]))
    t = pm.PageTables(2, 4, 8, 16)
    for bad in ((ints([1]), 5), (ints([1, 2]).long(), 5), (ints([1, 2]), -1), (ints([1, 2]), 2 ** 31), (ints([1, 2]).cpu(), 5), ([1, 2], 5)):
        with pytest.raises(ValueError):
            t.plan(*bad)
    with pytest.raises(ValueError):
        t.plan(ints([1, 2]), 5, keep=ints([1]))
    with pytest.raises(ValueError, match="stream"):
        class Elsewhere:
            device = torch.device("cuda", 99)
        cache.attend(q, tables, lens, stream=Elsewhere())


def test_tensors_moved_or_changed_since(pm):
    q, k, v, tables, lens = ref.case([20, 5], 4, 2, 64, 16, F16, F16)
    cache = pm.PagedKVCache.wrap(k, v)
    want = cache.attend(q, tables, lens)
    k.set_(k.clone())
    assert torch.equal(cache.attend(q, tables, lens), want)
    v.resize_(1, 2, 16, 64)
    with pytest.raises(ValueError, match="no longer"):
        cache.attend(q, tables, lens)
    t = pm.PageTables(2, 4, 8, 16)
    t.lens.resize_(1)
    with pytest.raises(ValueError, match="no longer"):
        t.plan(ints([1, 2]), 5)
