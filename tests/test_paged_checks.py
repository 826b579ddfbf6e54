"""What the paged KV cache operators refuse (no GPU needed: every refusal is made on the host before a launch)."""
import ctypes as C

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 7
P = 0x10000      # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def pm():
    import persistent_monokernel_gb300 as pm
    from persistent_monokernel_gb300 import build
    build.build()
    return pm


def cache(pm, **over):
    f = dict(n_pages=8, n_kv_heads=2, page=16, head_dim=128, dtype=0, k=P, v=4 * P, page_stride=4096, head_stride=2048,
             pos_stride=128)
    return pm.lf_paged(**{**f, **over})


def rows(pm, **over):
    return pm.lf_rows(**{**dict(data=P, dtype=0, token_stride=256, head_stride=128), **over})


CACHES = [(dict(n_pages=0), INVALID), (dict(n_kv_heads=0), INVALID), (dict(page=0), INVALID), (dict(page=-16), INVALID),
          (dict(head_dim=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
          (dict(n_kv_heads=1025), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
          (dict(n_pages=2 ** 27), UNSUPPORTED), (dict(k=0), INVALID), (dict(v=None), INVALID), (dict(k=P + 8), INVALID),
          (dict(v=P), INVALID), (dict(page_stride=4095), INVALID), (dict(page_stride=2048), INVALID),
          (dict(head_stride=128), INVALID), (dict(pos_stride=64), INVALID), (dict(pos_stride=-128), INVALID),
          (dict(pos_stride=0), INVALID), (dict(page_stride=2 ** 41), INVALID), (dict(pos_stride=256), INVALID)]


@pytest.mark.parametrize("over,status", CACHES)
def test_caches(pm, over, status):
    L, c, r, need = pm.lib(), cache(pm, **over), rows(pm), C.c_int64()
    assert L.lf_paged_append(C.byref(c), C.byref(r), C.byref(r), 1, P, None) == status
    q = pm.lf_paged_query(r, rows(pm, data=2 * P), 1, 2, P, 1, 1, P, 0, 0.0)
    assert L.lf_paged_workspace(C.byref(c), C.byref(q), C.byref(need)) == status
    assert L.lf_paged_attend(C.byref(c), C.byref(q), None, 0, None) == status


@pytest.mark.parametrize("over", [dict(head_stride=128, pos_stride=256), dict(page_stride=10000, head_stride=5000, pos_stride=136),
                                  dict(n_pages=1, page_stride=1), dict(n_kv_heads=1, head_stride=3)])
def test_strides_that_are_fine(pm, over):
    """Positions outside heads, gaps, and strides of dimensions of one; no rows, so that nothing is launched."""
    L, c, r = pm.lib(), cache(pm, **over), rows(pm)
    assert L.lf_paged_append(C.byref(c), C.byref(r), C.byref(r), 0, None, None) == OK


APPENDS = [(dict(n=-1), INVALID), (dict(slots=0), INVALID), (dict(slots=P + 2), INVALID), (dict(k=dict(data=0)), INVALID),
           (dict(k=dict(dtype=1)), INVALID), (dict(k=dict(dtype=1), v=dict(dtype=1)), INVALID), (dict(k=dict(dtype=3)), UNSUPPORTED),
           (dict(v=dict(token_stride=257)), INVALID), (dict(v=dict(head_stride=-128)), INVALID),
           (dict(k=dict(dtype=2)), INVALID), (dict(n=0), OK)]


@pytest.mark.parametrize("over,status", APPENDS)
def test_appends(pm, over, status):
    L, c = pm.lib(), cache(pm)
    k, v = rows(pm, **over.get("k", {})), rows(pm, **over.get("v", {}))
    assert L.lf_paged_append(C.byref(c), C.byref(k), C.byref(v), over.get("n", 2), over.get("slots", P), None) == status
    assert L.lf_paged_append(C.byref(c), None, C.byref(v), 2, P, None) == INVALID
    assert L.lf_paged_append(None, C.byref(k), C.byref(v), 2, P, None) == INVALID


QUERIES = [(dict(n_seqs=-1), INVALID), (dict(n_heads=0), INVALID), (dict(n_heads=3), UNSUPPORTED), (dict(table_width=-1), INVALID),
           (dict(table_stride=-1), INVALID), (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID),
           (dict(scale=float("-inf")), INVALID), (dict(table_width=2 ** 26 + 1), UNSUPPORTED),
           (dict(n_seqs=2 ** 26 + 1), UNSUPPORTED), (dict(q=dict(dtype=1)), INVALID), (dict(q=dict(dtype=5)), UNSUPPORTED),
           (dict(n_seqs=0), OK)]


@pytest.mark.parametrize("over,status", QUERIES)
def test_queries(pm, over, status):
    L, c, need = pm.lib(), cache(pm), C.c_int64(-1)
    f = dict(q=rows(pm, **over.get("q", {})), out=rows(pm, data=2 * P), n_seqs=2, n_heads=2, tables=P, table_stride=4,
             table_width=4, lens=P, window=0, scale=0.0)
    q = pm.lf_paged_query(**{**f, **{a: b for a, b in over.items() if a != "q"}})
    assert L.lf_paged_workspace(C.byref(c), C.byref(q), C.byref(need)) == status
    assert L.lf_paged_attend(C.byref(c), C.byref(q), None, 0, None) == status
    assert L.lf_paged_workspace(C.byref(c), C.byref(q), None) == INVALID
    assert L.lf_paged_attend(C.byref(c), None, None, 0, None) == INVALID
    if status == OK:
        assert need.value == 0


PLANS = [(dict(n_seqs=-1), INVALID), (dict(max_pages=0), INVALID), (dict(n_pages=0), INVALID), (dict(page=0), INVALID),
         (dict(page=40), UNSUPPORTED), (dict(n_seqs=8193, table_stride=4), UNSUPPORTED), (dict(n_pages=2 ** 27), UNSUPPORTED),
         (dict(max_pages=2 ** 26 + 1, table_stride=2 ** 27), UNSUPPORTED), (dict(table_stride=3), INVALID),
         (dict(table_stride=-4), INVALID), (dict(tables=0), INVALID), (dict(tables=P + 2), INVALID), (dict(lens=0), INVALID),
         (dict(free_pages=0), INVALID), (dict(n_free=None), INVALID), (dict(status=P + 1), INVALID)]
PLAN_ARGS = [(dict(n_new=0), INVALID), (dict(keep=P + 2), INVALID), (dict(slots=0), INVALID), (dict(slots=P + 4), INVALID),
             (dict(positions=P + 8), INVALID), (dict(offsets=0), INVALID), (dict(max_tokens=-1), INVALID),
             (dict(max_tokens=2 ** 30 + 1), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", PLANS + PLAN_ARGS)
def test_plans(pm, over, status):
    L = pm.lib()
    f = dict(n_seqs=2, max_pages=4, n_pages=8, page=16, tables=P, table_stride=4, lens=P, free_pages=P, n_free=P, status=P)
    t = pm.lf_page_tables(**{a: over.get(a, b) for a, b in f.items()})
    a = {**dict(n_new=P, keep=None, slots=P, positions=2 * P, offsets=P, max_tokens=64), **over}
    args = [a[x] for x in ("n_new", "keep", "slots", "positions", "offsets", "max_tokens")]
    assert L.lf_paged_plan(C.byref(t), *args, None) == status
    assert L.lf_paged_plan(None, *args, None) == INVALID


def test_structures_match_the_header(pm):
    import test_abi_layout as lay
    mine = ("lf_paged", "lf_page_tables", "lf_paged_query")
    keep, lay.STRUCTS = lay.STRUCTS, mine
    try:
        layout = lay._c_layout(pm)
    finally:
        lay.STRUCTS = keep
    for st in mine:
        cls = getattr(pm, st)
        assert layout[(st, "size")] == C.sizeof(cls)
        for name, _ in cls._fields_:
            assert layout[(st, name)] == getattr(cls, name).offset, (st, name)


def test_host_tensors_are_refused(pm):
    k, v = (torch.zeros(3, 2, 16, 64, dtype=torch.float16) for _ in range(2))
    with pytest.raises(ValueError, match="CUDA"):
        pm.PagedKVCache.wrap(k, v)
    with pytest.raises(ValueError, match="CUDA"):
        pm.PagedKVCache.wrap(k[0], v[0])
    ints = [torch.zeros(s, dtype=torch.int32) for s in ((2, 4), (2,), (8,), (1,))]
    with pytest.raises(ValueError, match="CUDA"):
        pm.PageTables.wrap(*ints, 16)
    for page in (0, 8, 40, -16):
        with pytest.raises(ValueError, match="multiple of 16"):
            pm.PageTables.wrap(*ints, page)


def test_tensors_have_no_setters(pm):
    for cls, names in ((pm.PagedKVCache, ("k", "v")), (pm.PageTables, ("tables", "lens", "free", "n_free", "status"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(cls.__new__(cls), name, None)
