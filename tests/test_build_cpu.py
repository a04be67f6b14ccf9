"""The build of the library and of the bindings' native checks, which are bound to the installed torch and may be
missing without taking the library along (CPU only)."""
import os

import pytest
import torch

from paged_kv_cache_62_gb300 import build as pkv_build
from paged_kv_cache_62_gb300 import pkv


@pytest.fixture
def torch_part(tmp_path, monkeypatch):
    """The library is built; the paths of the torch part lie in a folder of their own."""
    pkv_build.build()
    path = {}
    for name in ("TORCH_PATH", "TORCH_OBJ", "TORCH_KEY"):
        path[name] = str(tmp_path / name.lower())
        monkeypatch.setattr(pkv_build, name, path[name], raising=False)
    return path


def commands(torch_part, calls, ok=True):
    def f(*a):
        calls.append(1)
        if not ok:
            return ["false"], ["false"]
        return ["touch", torch_part["TORCH_OBJ"]], ["touch", a[-1]]
    return f


@pytest.mark.parametrize("how", ["compiler", "no torch", "no g++"])
def test_the_library_is_built_where_the_torch_part_fails(torch_part, monkeypatch, capfd, how):
    with open(torch_part["TORCH_PATH"], "w") as f:
        f.write("an old one")

    def missing(*a):
        raise ImportError("no torch here")

    monkeypatch.setattr(pkv_build, "torch_commands", {"compiler": commands(torch_part, [], False), "no torch": missing,
                                                      "no g++": lambda *a: (["/no/such/compiler"],) * 2}[how])
    assert pkv_build.build() == pkv_build.LIB_PATH
    assert os.path.exists(pkv_build.LIB_PATH)
    assert not os.path.exists(torch_part["TORCH_PATH"])         # nothing stale is left to be loaded
    assert "_pkv_torch.so was not built" in capfd.readouterr().err
    pkv.load()


def test_the_torch_part_follows_the_installed_torch(torch_part, monkeypatch):
    calls = []
    monkeypatch.setattr(pkv_build, "torch_commands", commands(torch_part, calls))
    pkv_build.build()
    assert os.path.exists(torch_part["TORCH_PATH"]) and calls
    calls.clear()
    pkv_build.build()
    assert not calls                                            # up to date
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    pkv_build.build()
    assert calls
    calls.clear()
    pkv_build.build()
    assert not calls


def test_a_torch_part_of_another_torch_is_refused(monkeypatch):
    pkv_build.build()
    monkeypatch.setattr(pkv, "_torch_native", None)
    assert pkv._native().torch_version == torch.__version__
    monkeypatch.setattr(pkv, "_torch_native", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    with pytest.raises(RuntimeError, match="built for torch"):
        pkv._native()
    with pytest.raises(RuntimeError, match="built for torch"):
        pkv.copy_blocks_i8(None, None, None, None)
