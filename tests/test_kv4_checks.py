"""What the 4-bit KV cache operators refuse (no GPU needed: every refusal is made on the host before a launch)."""
import ctypes as C
import os

import pytest
import torch

from conftest import ROOT

OK, INVALID, CAPACITY, UNSUPPORTED = 0, 1, 3, 7
P = 0x10000      # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def pm():
    import persistent_monokernel_gb300 as pm
    from persistent_monokernel_gb300 import build
    build.build()
    return pm


def cache(pm, **over):
    f = dict(n_kv_heads=2, head_dim=128, max_seq=64, k_codes=P, k_scales=P, v_codes=P, v_scales=P)
    return pm.lf_kv4(**{**f, **over})


def rows(pm, **over):
    return pm.lf_rows(**{**dict(data=P, dtype=0, token_stride=256, head_stride=128), **over})


CACHES = [(dict(n_kv_heads=0), INVALID), (dict(max_seq=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
          (dict(head_dim=256), UNSUPPORTED), (dict(n_kv_heads=1025), UNSUPPORTED), (dict(max_seq=2 ** 30 + 1), UNSUPPORTED), (dict(k_codes=0), INVALID),
          (dict(v_scales=P + 8), INVALID), (dict(v_codes=P + 4), INVALID), (dict(k_scales=None), INVALID)]


@pytest.mark.parametrize("over,status", CACHES)
def test_caches(pm, over, status):
    L, c, r, need = pm.lib(), cache(pm, **over), rows(pm), C.c_int64()
    for f in (L.lf_kv4_append, L.lf_kv4_read):
        assert f(C.byref(c), C.byref(r), C.byref(r), 1, 0, None) == status
    q = pm.lf_kv4_query(r, rows(pm, data=2 * P), 2, 1, 0, 1, 0, 0.0)
    assert L.lf_kv4_workspace(C.byref(c), C.byref(q), C.byref(need)) == status
    assert L.lf_kv4_attend(C.byref(c), C.byref(q), None, 0, None) == status


@pytest.mark.parametrize("n,pos,status", [(-1, 0, INVALID), (1, -1, INVALID), (1, 64, CAPACITY), (65, 0, CAPACITY),
                                          (2 ** 31 - 1, 2 ** 31 - 1, CAPACITY), (0, 0, OK), (0, 64, OK), (0, 65, CAPACITY)])
def test_positions(pm, n, pos, status):
    L, c, r = pm.lib(), cache(pm), rows(pm)
    for f in (L.lf_kv4_append, L.lf_kv4_read):
        assert f(C.byref(c), C.byref(r), C.byref(r), n, pos, None) == status


ROWS = [(dict(data=0), INVALID), (dict(data=P + 2), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
        (dict(token_stride=-256), INVALID), (dict(token_stride=257), INVALID), (dict(head_stride=132), INVALID),
        (dict(token_stride=1 << 41), INVALID)]


@pytest.mark.parametrize("over,status", ROWS)
def test_rows(pm, over, status):
    L, c, good, bad = pm.lib(), cache(pm), rows(pm), rows(pm, **over)
    for f in (L.lf_kv4_append, L.lf_kv4_read):
        assert f(C.byref(c), C.byref(bad), C.byref(good), 2, 0, None) == status
        assert f(C.byref(c), C.byref(good), C.byref(bad), 2, 0, None) == status
        assert f(C.byref(c), None, C.byref(good), 2, 0, None) == INVALID
        assert f(None, C.byref(good), C.byref(good), 2, 0, None) == INVALID


@pytest.mark.parametrize("over", [dict(token_stride=0), dict(token_stride=128), dict(head_stride=0), dict(head_stride=64)])
def test_tensors_that_are_written_must_not_overlap_themselves(pm, over):
    L, c, good, bad = pm.lib(), cache(pm), rows(pm), rows(pm, **over)
    assert L.lf_kv4_read(C.byref(c), C.byref(good), C.byref(bad), 2, 0, None) == INVALID


def test_k_and_v_of_one_dtype(pm):
    L, c = pm.lib(), cache(pm)
    a, b = rows(pm), rows(pm, dtype=1)
    assert L.lf_kv4_append(C.byref(c), C.byref(a), C.byref(b), 1, 0, None) == INVALID
    assert L.lf_kv4_read(C.byref(c), C.byref(a), C.byref(b), 1, 0, None) == INVALID


QUERIES = [(dict(n_heads=0), INVALID), (dict(n_heads=3), UNSUPPORTED), (dict(n=-1), INVALID), (dict(pos=-1), INVALID),
           (dict(length=-1), INVALID), (dict(length=65), CAPACITY), (dict(window=-1), INVALID),
           (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
           (dict(n=1 << 28, n_heads=4), UNSUPPORTED), (dict(pos=2 ** 31 - 5), UNSUPPORTED), (dict(pos=2 ** 30 - 1), UNSUPPORTED), (dict(n=0), OK)]


@pytest.mark.parametrize("over,status", QUERIES)
def test_queries(pm, over, status):
    L, c, need = pm.lib(), cache(pm), C.c_int64(-1)
    f = dict(q=rows(pm), out=rows(pm, data=2 * P), n_heads=2, n=2, pos=0, length=2, window=0, scale=0.0)
    q = pm.lf_kv4_query(**{**f, **over})
    assert L.lf_kv4_workspace(C.byref(c), C.byref(q), C.byref(need)) == status
    assert L.lf_kv4_attend(C.byref(c), C.byref(q), None, 0, None) == status
    assert L.lf_kv4_workspace(C.byref(c), C.byref(q), None) == INVALID
    assert L.lf_kv4_attend(C.byref(c), None, None, 0, None) == INVALID
    assert L.lf_kv4_attend(None, C.byref(q), None, 0, None) == INVALID
    if status == OK:
        assert need.value == 0


def test_k_and_v_are_read_to_different_places(pm):
    L, c, r = pm.lib(), cache(pm), rows(pm)
    assert L.lf_kv4_read(C.byref(c), C.byref(r), C.byref(r), 1, 0, None) == INVALID


def test_rows_of_all_heads_are_counted_in_64_bits(pm):
    L, c, need = pm.lib(), cache(pm, n_kv_heads=1024), C.c_int64(-1)
    r = rows(pm, token_stride=0, head_stride=0)
    for n, heads in (((1 << 22) + 1, 1024), (1 << 28, 1024), (1 << 18, 16385 * 1024)):
        q = pm.lf_kv4_query(r, rows(pm, data=2 * P), heads, n, 0, 1, 0, 0.0)
        assert L.lf_kv4_workspace(C.byref(c), C.byref(q), C.byref(need)) == UNSUPPORTED
        assert L.lf_kv4_attend(C.byref(c), C.byref(q), 3 * P, 1 << 40, None) == UNSUPPORTED


def test_structures_match_the_header(pm):
    import test_abi_layout as lay
    mine = ("lf_kv4", "lf_rows", "lf_kv4_query")
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


def test_constants_match_the_header():
    from persistent_monokernel_gb300 import kv4
    text = open(os.path.join(ROOT, "include", "lf.h")).read()
    for name, val in (("LF_F16", kv4.F16), ("LF_BF16", kv4.BF16), ("LF_F32", kv4.F32)):
        assert f"#define {name} {val}\n" in text


def test_host_tensors_are_refused(pm):
    z = [torch.zeros(2, 8, w, dtype=torch.uint8) for w in (32, 4, 32, 4)]
    with pytest.raises(ValueError, match="CUDA"):
        pm.KV4Cache.wrap(*z)
    with pytest.raises(ValueError):
        pm.KV4Cache.wrap(z[0][0], *z[1:])


def test_a_decoder_on_the_4_bit_cache_checks_its_arguments_like_lf_create(pm):
    L, h = pm.lib(), C.c_void_p()
    w = pm.lf_weights(*([0x1000] * 12))
    good = dict(n_layers=2, d_model=256, n_heads=4, n_kv_heads=4, head_dim=64, ffn_dim=1024, vocab=4096, max_seq=64,
                rope_theta=10000.0, rms_eps=1e-5, fault_step=-1)
    for change, status in ((dict(head_dim=96), UNSUPPORTED), (dict(max_seq=0), INVALID), (dict(prefill_block=-2), INVALID)):
        cfg = pm.lf_config(**{**good, **change})
        assert L.lf_create_kv4(C.byref(cfg), C.byref(w), C.byref(h)) == status
    assert L.lf_create_kv4(None, C.byref(w), C.byref(h)) == INVALID
