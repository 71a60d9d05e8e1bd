"""The optional extensions: one that does not compile, does not load or was built for another torch is
left out with a warning, and the binding's Python code makes the same calls."""
import os
import types

import pytest

from prefix_cached_kv_radix_gb300 import api, build


@pytest.fixture
def out(tmp_path, monkeypatch):
    """Path of _rxops in a build folder of the test's own, and the compilers' calls."""
    if build.build_pyops() is None:
        pytest.skip("no headers to build the extension against")
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    return build.pystep_path("_rxops")


def touch(path):
    with open(path, "w") as f:
        f.write("not an extension")


def test_extension_that_does_not_compile_is_left_out(out, monkeypatch):
    def fails(cmd, verbose):
        raise RuntimeError("build failed")
    monkeypatch.setattr(build, "_run", fails)
    touch(out)
    with pytest.warns(UserWarning, match="does not compile"):
        assert build.build_pyops() is None
    assert not os.path.exists(out)                         # an old one is not left to be loaded
    assert api._load_ext("_rxops") is False


def test_extension_is_built_anew_for_another_torch(out, monkeypatch):
    calls = []

    def compiles(cmd, verbose):
        calls.append(cmd)
        touch(cmd[cmd.index("-o") + 1])
    monkeypatch.setattr(build, "_run", compiles)
    assert build.build_pyops() == out and build.build_pyops() == out and len(calls) == 1
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert build.build_pyops() == out and len(calls) == 2


@pytest.mark.parametrize("name", ["_rxops", "_rxstep"])
def test_extension_that_does_not_load_is_left_out(out, name):
    touch(build.pystep_path(name))
    with pytest.warns(UserWarning, match="does not load"):
        assert api._load_ext(name) is False


def test_extension_for_another_torch_is_not_used(monkeypatch):
    monkeypatch.setattr(api, "_ops_ext", None)
    monkeypatch.setattr(api, "_load_ext", lambda name: types.SimpleNamespace(torch_version="0.0.1", bind=None))
    with pytest.warns(UserWarning, match="built for torch 0.0.1"):
        assert api.ops_ext() is None
    assert api._ops_ext is False                           # decided once


def test_extension_of_this_build_is_used(monkeypatch):
    if not os.path.exists(build.pystep_path("_rxops")):
        pytest.skip("not built")
    monkeypatch.setattr(api, "_ops_ext", None)
    ext = api.ops_ext()
    assert ext is not None and all(hasattr(ext, n) for n in ("kv_pool_write_rope", "kv_pool_copy", "kv_pool_fork", "prompt_attention"))
