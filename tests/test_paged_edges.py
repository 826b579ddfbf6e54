"""The paged KV cache's host side where it can go wrong (no GPU needed)."""
import pytest
import torch


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
