"""Building: the library comes without torch or the Python headers, as a C program needs it."""
import importlib.util
import os
import shutil
import sys
import sysconfig

import pytest

import bit_mla_kv_qcache_gb300.build as package_build


@pytest.fixture
def recipe(tmp_path, monkeypatch):
    """A copy of the build recipe that makes one small source's library in a folder of its own."""
    if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no nvcc")
    spec = importlib.util.spec_from_file_location("recipe", package_build.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(m, "SOURCES", {"diag.cu": []})
    for name, value in (("BUILD", tmp_path / "obj"), ("LIB", tmp_path / "lib.so"), ("FAST", tmp_path / "fast.so"), ("PKG", tmp_path)):
        monkeypatch.setattr(m, name, str(value))
    return m


@pytest.mark.parametrize("missing", ["torch", "headers"])
def test_the_library_is_built_without(recipe, monkeypatch, tmp_path, missing):
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.warns(UserWarning, match="native binding"):
        assert recipe.build() == recipe.LIB
    assert os.path.exists(recipe.LIB) and not os.path.exists(recipe.FAST)
    before = os.path.getmtime(recipe.LIB)
    with pytest.warns(UserWarning, match="native binding"):
        recipe.build()
    assert os.path.getmtime(recipe.LIB) == before  # not made again


def test_a_binding_that_does_not_compile_is_an_error(recipe, monkeypatch, tmp_path):
    bad = tmp_path / "fastcall.cpp"
    bad.write_text("not C++\n")
    monkeypatch.setattr(recipe, "FAST_SOURCE", str(bad))
    with pytest.raises(RuntimeError, match="fastcall"):
        recipe.build()
    assert os.path.exists(recipe.LIB)  # and a C program has its library
