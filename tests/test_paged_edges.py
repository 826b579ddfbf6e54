"""The paged KV cache's host side where it can go wrong (no GPU needed)."""
import pytest
import torch

from paged_launch import launches


@pytest.fixture(scope="module")
def pm():
    import persistent_monokernel_gb300 as pm
    from persistent_monokernel_gb300 import build
    build.build()
    return pm


@pytest.mark.parametrize("args", [(4, 2, 64, 8), (4, 2, 96), (0, 2, 64), (4, 0, 64), (4, 1025, 64), (2 ** 27, 1, 64), (4, 2, 64, 24),
                                  (4, 2, 64, 0), (4, -2, 64), (2 ** 30, 2 ** 10, 128)])
def test_pools_that_cannot_be_are_refused_at_once(pm, args):
    """Before any memory is asked for: the last one's would be 10^16 bytes."""
    with pytest.raises(pm.LFError):
        pm.PagedKVCache(*args)


def test_sizes_and_types_that_cannot_be(pm):
    for args, dtype in (((4, 2, 64, 2 ** 31), None), ((2 ** 32 + 4, 2, 64), None), ((4, 2, 64), torch.float32), ((4, 2, 64), torch.int8)):
        with pytest.raises(ValueError):
            pm.PagedKVCache(*args, dtype=dtype)


# ---------------------------------------------------------------- the attention's launches

PLACES = 304                                               # CTAs of four warps that 152 SMs hold


def test_many_rows_get_no_more_ctas_than_they_use(tmp_path):
    """With more sequences and heads than fit at a time, clusters multiply rounds of CTAs whose rows may be short: at most
    eight rounds of them, and single CTAs where there are more already, however wide the table is."""
    shapes = [(n, group, hkv, hd, page, width // page, window)
              for n in (1, 2, 200, 256, 257, 300, 450, 600, 1000, 5000) for group, hkv in ((4, 8), (4, 5), (16, 2), (17, 1), (8, 1), (1, 40))
              for hd in (64, 128) for page in (16, 64) for width in (64, 1024, 4096, 8192, 32768, 131072, 2 ** 20) for window in (0, 1000, 20000)]
    for (n, group, hkv, *_, window), got in zip(shapes, launches(shapes, str(tmp_path))):
        items = n * hkv * (2 if group == 17 else 1)
        if items > PLACES:
            assert got.parts == 1 and (got.cl == 1 or items * got.cl <= 8 * PLACES), (n, group, hkv, got)


@pytest.mark.parametrize("width", [1024, 4096, 16384, 32768, 131072])
def test_launches_of_a_row_more(tmp_path, width):
    """256 rows can be sorted by length and 257 are not: that is all that changes for eight KV heads."""
    few, *more = launches([(n, 4, 8, 128, 64, width // 64, 0) for n in (256, 257, 300, 1000)], str(tmp_path))
    for got in more:
        assert got == few._replace(sorted=0) and got.cl == 1


def test_launches_that_the_rule_describes(tmp_path):
    """A launch of each kind (rows, heads per KV head, KV heads, head_dim, page, columns, window)."""
    kinds = [((1, 4, 5, 128, 64, 8, 0), (4, 4, 1, 0)), ((1, 4, 5, 128, 64, 128, 0), (8, 8, 1, 0)), ((1, 4, 5, 128, 64, 512, 0), (4, 4, 14, 0)),
             ((24, 4, 5, 128, 64, 47, 0), (2, 4, 1, 0)), ((16, 4, 8, 128, 64, 512, 0), (8, 4, 1, 1)), ((64, 4, 8, 128, 64, 256, 0), (2, 4, 1, 1)),
             ((200, 16, 2, 128, 48, 417, 0), (4, 4, 1, 1)), ((64, 4, 8, 128, 64, 64, 0), (1, 4, 1, 1)), ((600, 16, 2, 128, 64, 64, 0), (2, 4, 1, 0)),
             ((257, 16, 2, 128, 64, 256, 0), (4, 4, 1, 0)), ((280, 8, 1, 128, 64, 1024, 0), (8, 4, 1, 0))]
    assert launches([q for q, _ in kinds], str(tmp_path)) == [want for _, want in kinds]
