"""What the 4-bit KV cache's Python side does without a GPU."""
import pytest


def test_a_caches_tensors_have_no_setters():
    """The calls use the tensors that the cache was made with: one in their place would be ignored."""
    from persistent_monokernel_gb300 import KV4Cache
    cache = KV4Cache.__new__(KV4Cache)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        with pytest.raises(AttributeError):
            setattr(cache, name, None)


class _Cuda:
    """As much of torch.cuda as KV4Cache.sync asks for."""
    def device(self, d):
        import contextlib
        return contextlib.nullcontext()

    def current_stream(self):
        import types
        return types.SimpleNamespace(cuda_stream=0)


def test_every_cache_is_told_of_a_wait_that_ran_out(monkeypatch):
    """The library tells once for the device: the cache that asks first must not keep it from the others."""
    import types

    from persistent_monokernel_gb300 import KV4Cache, kv4
    answers = []
    monkeypatch.setattr(kv4, "_torch", types.SimpleNamespace(cuda=_Cuda()))
    monkeypatch.setattr(kv4, "_lib", types.SimpleNamespace(lf_kv4_status=lambda s: answers.pop(0) if answers else 0))

    def cache(device):
        c = KV4Cache.__new__(KV4Cache)
        c.device, c._heard = device, getattr(kv4, "_told", {}).get(device, 0)
        return c

    a, b, other = cache("x"), cache("x"), cache("y")
    assert a.sync() == b.sync() == 0
    answers.append(6)
    assert [a.sync(), b.sync(), other.sync()] == [6, 6, 0]
    assert [a.sync(), b.sync(), other.sync(), cache("x").sync()] == [0, 0, 0, 0]
    answers.append(5)                                     # another error is neither remembered nor mistaken
    assert [b.sync(), a.sync(), b.sync()] == [5, 0, 0]
    answers += [6, 6]
    assert [b.sync(), b.sync(), b.sync(), a.sync(), a.sync()] == [6, 6, 0, 6, 0]
