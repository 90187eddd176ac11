"""What is built when: the library with nvcc alone, the torch-facing module beside it
only for the torch that is installed; and calls without that module."""
import os
import warnings

import pytest

import bit_quantized_tensor_gb300 as qg
from bit_quantized_tensor_gb300 import _build
from tests.test_block_host import Library, Stream, Torch, calls


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A build into tmp_path with compilers that only write their output; returns what ran."""
    ran = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        ran.append("host" if "_qg_host" in out else "link" if "libqgemm" in out else "compile")
        with open(out, "w"):
            pass
        return type("Done", (), dict(returncode=0, stdout="", stderr=""))

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    for name, file in (("BUILD_DIR", "build"), ("LIB", "libqgemm.so"), ("HOST", "_qg_host.so"), ("HOST_FOR", "build/for")):
        monkeypatch.setattr(_build, name, str(tmp_path / file))
    monkeypatch.setattr(_build, "_installed", lambda: "torch 2, Python 3")
    return ran


def test_each_is_built_when_it_is_out_of_date(tree, monkeypatch):
    _build.build()
    assert tree.count("host") == tree.count("link") == 1 and tree.count("compile") == len(_build.sources())
    tree.clear()
    assert _build.up_to_date()
    _build.build()
    assert tree == []
    monkeypatch.setattr(_build, "_installed", lambda: "torch 3, Python 3")  # another torch: the module alone
    assert not _build.up_to_date()
    _build.build()
    assert tree == ["host"] and _build.up_to_date()
    os.remove(_build.HOST)
    assert not _build.up_to_date()
    os.remove(_build.LIB)
    tree.clear()
    _build.build()
    assert tree.count("host") == tree.count("link") == 1


def test_the_library_builds_without_torch(tree, monkeypatch):
    monkeypatch.setattr(_build, "_installed", lambda: "")
    _build.build()
    assert "host" not in tree and tree.count("link") == 1 and _build.up_to_date()


def test_a_module_that_does_not_build_leaves_the_library(tree, monkeypatch):
    def fails():
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(_build, "build_host", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        _build.build()
    assert os.path.exists(_build.LIB) and not _build.up_to_date()


def test_calls_without_the_module(monkeypatch):
    """They say so once and go through ctypes."""
    import sys
    torch, lib = Torch(), Library()
    monkeypatch.setattr(qg, "_torch_module", torch)
    monkeypatch.setattr(qg, "lib", lambda: lib)
    monkeypatch.setattr(qg, "_dtype_ids", None)
    monkeypatch.setattr(qg, "_host_module", None)
    monkeypatch.delattr(qg, "_qg_host", raising=False)
    monkeypatch.setitem(sys.modules, qg.__name__ + "._qg_host", None)
    with warnings.catch_warnings(record=True) as seen:
        warnings.simplefilter("always")
        for name, call in calls(torch).items():
            call(stream=Stream(2))
            assert lib.launched[-1] == (name, 2)
    assert [w.category for w in seen] == [RuntimeWarning] and "_qg_host.so is missing" in str(seen[0].message)
