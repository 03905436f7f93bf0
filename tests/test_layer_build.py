"""The build's two products: the library, which needs nvcc only, and the Python binding of the
layer operators, which needs the torch it is loaded into.  On a one-function library."""
import ctypes
import os
import subprocess
import sys
import types

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


def _torch(root, version, value):
    """A stand-in for an installed torch: a header that says which, and libraries to link."""
    at = root / version
    (at / "include").mkdir(parents=True)
    (at / "lib").mkdir()
    (at / "include" / "which.h").write_text(f"#define WHICH {value}\n")
    for name in ("torch_python", "torch_cpu", "c10", "c10_cuda"):
        subprocess.run(["gcc", "-shared", "-x", "c", "/dev/null", "-o", str(at / "lib" / f"lib{name}.so")], check=True)
    fake = types.ModuleType("torch")
    fake.__version__, fake.__file__ = version, str(at / "__init__.py")
    fake._C = types.SimpleNamespace(_GLIBCXX_USE_CXX11_ABI=True)
    return fake


def test_each_torch_loads_the_binding_built_for_it(tree, monkeypatch):
    """Back and forth between two versions, with what the first build left lying there."""
    fakes = {1: _torch(tree, "1.0", 1), 2: _torch(tree, "2.0", 2)}
    for value in (1, 2, 1, 2):
        monkeypatch.setitem(sys.modules, "torch", fakes[value])
        m2build.build()
        code = f"import ctypes; print(ctypes.CDLL({m2build.ext_path()!r}).which())"     # a process each: loaded once by name
        assert int(subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, check=True).stdout) == value


def test_warnings_about_the_binding_are_shown(tree, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", _torch(tree, "1.0", 1))
    m2build.build()
    assert capsys.readouterr().err == ""
    (tree / "binding" / "layer_ext.cpp").write_text("int f() { int unused; return 1; }\n")
    m2build.build(force=True)
    assert "unused" in capsys.readouterr().err
