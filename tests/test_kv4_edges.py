"""What the 4-bit KV cache's Python side does without a GPU."""
import os
import types

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


# ---------------------------------------------------------------- the build

@pytest.fixture
def shop(monkeypatch, tmp_path):
    """build.py with compilers that write empty files, or fail for what `broken` names."""
    from persistent_monokernel_gb300 import build
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'\n")
    s = types.SimpleNamespace(build=build, ran=[], broken=None, torch=torch, have_torch=True)

    def run(cmd, **k):
        s.ran.append(cmd)
        if s.broken and any(s.broken in c for c in cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: types.SimpleNamespace(
        submodule_search_locations=[str(torch)]) if s.have_torch else None)
    for name, value in (("LIB", "liblf.so"), ("EXT", "_lft.so"), ("BUILD", "_build")):
        monkeypatch.setattr(build, name, str(tmp_path / value))
    return s


def test_the_library_is_built_without_torch(shop):
    shop.have_torch = False
    assert shop.build.build() == shop.build.LIB
    assert os.path.exists(shop.build.LIB) and not os.path.exists(shop.build.EXT)
    assert shop.build.up_to_date()
    shop.build.build(force=True)


def test_the_library_stands_where_the_module_of_calls_cannot_be_built(shop):
    shop.broken = "lf_torch.cpp"
    with pytest.raises(RuntimeError, match="lf_torch.cpp"):
        shop.build.build()
    assert os.path.exists(shop.build.LIB) and not shop.build.up_to_date()


def test_another_torch_gets_another_module_of_calls(shop):
    shop.build.build()
    assert shop.build.up_to_date()
    (shop.torch / "version.py").write_text("__version__ = '2'\n")
    assert not shop.build.up_to_date()
    shop.ran.clear()
    shop.build.build()
    assert shop.build.up_to_date() and [any("lf_torch.cpp" in c for c in cmd) for cmd in shop.ran] == [True]


def test_a_module_of_calls_for_another_torch_is_not_used(monkeypatch):
    """(A tree that was built, then met another torch or Python without being built again.)"""
    import sys

    import persistent_monokernel_gb300 as pm
    from persistent_monokernel_gb300 import kv4
    monkeypatch.setattr(pm, "lib", lambda: types.SimpleNamespace())
    for made in (("0.9.0", sys.hexversion >> 16), (None, 0x309)):
        import torch
        fake = types.SimpleNamespace(made_for=(made[0] or torch.__version__.split("+")[0], made[1]))
        monkeypatch.setitem(sys.modules, "persistent_monokernel_gb300._lft", fake)
        monkeypatch.setattr(pm, "_lft", fake, raising=False)
        with pytest.raises(ImportError, match="built for torch"):
            kv4._load()
