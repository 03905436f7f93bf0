"""The build's two products: the library, which needs nvcc only, and the Python binding of the
layer operators, which needs the torch it is loaded into.  On a one-function library."""
import ctypes
import os
import sys

import pytest

from mamba_ssd_chunked_02_gb300 import build as m2build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build's folders moved to an empty place, with a small source of each kind."""
    for d in ("csrc", "include", "binding"):
        (tmp_path / d).mkdir()
    (tmp_path / "csrc" / "one.cu").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    ext = tmp_path / "binding" / "layer_ext.cpp"
    ext.write_text('#include <which.h>\nextern "C" __attribute__((visibility("default"))) int which() { return WHICH; }\n')
    lib = tmp_path / "_lib"
    for name, at in dict(CSRC=tmp_path / "csrc", INCLUDE=tmp_path / "include", BUILD=tmp_path / "_build", LIBDIR=lib,
                         LIB=lib / "libmamba2_ssd.so", EXT_SRC=ext).items():
        monkeypatch.setattr(m2build, name, str(at))
    monkeypatch.setattr(m2build, "EXT", str(lib / "layer_ext.so"), raising=False)
    return tmp_path


def test_the_library_is_built_without_torch(tree, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)      # import torch raises ImportError
    assert ctypes.CDLL(m2build.build()).one() == 1
    assert "torch" in capsys.readouterr().err
    assert [n for n in os.listdir(tree / "_lib") if "ext" in n] == []


def test_the_library_is_built_when_the_binding_does_not_compile(tree):
    (tree / "binding" / "layer_ext.cpp").write_text("#error no\n")
    with pytest.raises(RuntimeError, match="layer_ext.cpp"):
        m2build.build()
    assert ctypes.CDLL(m2build.LIB).one() == 1
