"""What the 4-bit KV cache's Python side does without a GPU."""
import pytest


def test_a_caches_tensors_have_no_setters():
    """The calls use the tensors that the cache was made with: one in their place would be ignored."""
    from persistent_monokernel_gb300 import KV4Cache
    cache = KV4Cache.__new__(KV4Cache)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        with pytest.raises(AttributeError):
            setattr(cache, name, None)
