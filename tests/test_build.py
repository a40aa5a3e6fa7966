"""build.py: the library does not depend on the binding's marshalling, and a marshalling of another interpreter, torch or
older sources does not stay. The compilers are replaced by one that only makes its output file."""
import os
import pathlib
import subprocess
import warnings

import pytest

from compressed_sparse_attention_append_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs under a folder of their own; returns the outputs' names, the compilers run and those that fail."""
    calls, broken = [], set()

    def check_call(cmd, **kw):
        tool = "nvcc" if "nvcc" in os.path.basename(cmd[0]) else "g++"
        calls.append(tool)
        if tool in broken:
            raise subprocess.CalledProcessError(1, cmd)
        pathlib.Path(cmd[cmd.index("-o") + 1]).write_text(tool)

    lib, marshal = str(tmp_path / "libcsa2.so"), str(tmp_path / "_marshal.x.so")
    monkeypatch.setattr(build, "LIB", lib)
    monkeypatch.setattr(build, "MARSHAL", marshal)
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    return lib, marshal, calls, broken


def test_the_library_is_built_without_the_marshalling(tree):
    lib, marshal, calls, broken = tree
    broken.add("g++")
    with pytest.warns(UserWarning, match="marshalling is not built"):
        assert build.build() == lib
    assert os.path.exists(lib) and not os.path.exists(marshal)


def test_a_missing_torch_leaves_the_library(tree, monkeypatch):
    lib, marshal, calls, broken = tree
    monkeypatch.setitem(__import__("sys").modules, "torch", None)  # (import torch raises ImportError)
    with pytest.warns(UserWarning, match="marshalling is not built"):
        build.build()
    assert os.path.exists(lib) and calls == ["nvcc"]


def test_a_failing_library_build_fails(tree):
    tree[3].add("nvcc")
    with pytest.raises(subprocess.CalledProcessError):
        build.build()


def test_nothing_is_built_twice_and_a_change_of_abi_or_sources_rebuilds(tree, tmp_path):
    lib, marshal, calls, broken = tree
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        build.build()
        assert calls == ["nvcc", "g++"] and os.path.exists(marshal)
        build.build()
        assert calls == ["nvcc", "g++"]
        pathlib.Path(marshal + ".abi").write_text("cpython-99 torch 1.0 cxx11 1")
        build.build()
        assert calls == ["nvcc", "g++", "g++"]
        os.utime(marshal, (1, 1))  # older than its source
        build.build()
        assert calls == ["nvcc", "g++", "g++", "g++"]
    # a build that fails leaves none of the old module
    (tmp_path / "_marshal.so").write_text("of any interpreter")
    os.utime(marshal, (1, 1))
    broken.add("g++")
    with pytest.warns(UserWarning):
        build.build()
    assert not os.path.exists(marshal) and not os.path.exists(tmp_path / "_marshal.so")
    assert os.path.exists(lib)


def test_the_module_is_named_for_its_interpreter():
    import importlib.machinery

    assert build.MARSHAL.endswith(importlib.machinery.EXTENSION_SUFFIXES[0])
