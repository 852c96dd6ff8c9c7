"""Building the library and the binding's extension module (without a GPU; nvcc is a stand-in)."""
import importlib.machinery
import os
import sys
import warnings

import pytest

torch = pytest.importorskip("torch")

from long_context_sparse_index_gb300 import build as b

NVCC = """#!/bin/sh
while [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo built > "$2"; fi; shift; done
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build into an empty folder, by an nvcc that only writes its output."""
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(NVCC)
    nvcc.chmod(0o755)
    monkeypatch.setattr(b, "_nvcc", lambda: str(nvcc))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libdsa.so"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "MARSHAL", str(tmp_path / os.path.basename(b.MARSHAL)))
    return tmp_path


@pytest.mark.parametrize("how", ["it fails", "no compiler", "no torch"])
def test_library_is_built_without_the_extension_module(tree, monkeypatch, how):
    """A clean tree and one whose library is up to date: the library stands, a warning says why the module does not, and
    none of an earlier build is left to be loaded."""
    if how == "no torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setenv("CXX", "false" if how == "it fails" else str(tree / "none"))
    for _ in range(2):
        for old in (b.MARSHAL, str(tree / "_marshal.so")):
            with open(old, "w") as f:
                f.write("of another build")
        with pytest.warns(RuntimeWarning, match="extension module was not built"):
            assert b.build() == b.LIB
        assert os.path.exists(b.LIB) and not any("_marshal" in n for n in os.listdir(tree))


def test_two_builds_at_once(tree, monkeypatch):
    """What one of them removes is gone for the other one, which goes on."""
    real = os.remove

    def late(path):
        real(path)
        raise FileNotFoundError(path)

    monkeypatch.setattr(os, "remove", late)
    monkeypatch.setenv("CXX", "false")
    for name in ("_marshal.so", os.path.basename(b.MARSHAL)):
        (tree / name).write_text("of another build")
    with pytest.warns(RuntimeWarning, match="was not built"):
        b.build()
    assert not any("_marshal" in n for n in os.listdir(tree))


def test_extension_module_is_built_beside_the_library(tree, monkeypatch):
    """Also where the library is up to date, and for each torch anew; no warning."""
    compiler = tree / "cxx"
    compiler.write_text(NVCC)
    compiler.chmod(0o755)
    monkeypatch.setenv("CXX", str(compiler))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        b.build()
        assert os.path.exists(b.MARSHAL)
        os.remove(b.MARSHAL)
        b.build()
        assert os.path.exists(b.MARSHAL)
        at = os.stat(b.MARSHAL).st_mtime_ns
        b.build()
        assert os.stat(b.MARSHAL).st_mtime_ns == at
        monkeypatch.setattr(torch, "__version__", "0.0")
        os.utime(b.MARSHAL, ns=(at + 10 ** 9, at + 10 ** 9))
        b.build()
        assert os.stat(b.MARSHAL).st_mtime_ns != at + 10 ** 9


def test_extension_module_is_for_this_python():
    """Its name is one that no other Python imports."""
    suffix = b.MARSHAL[b.MARSHAL.index("_marshal") + len("_marshal"):]
    assert suffix == importlib.machinery.EXTENSION_SUFFIXES[0] != ".so"
