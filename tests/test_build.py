"""The build of the library and of the Python module beside it, with small sources in a folder of their own (CPU)."""
import os
import shutil
import subprocess
import sys

import pytest

LIBRARY = "extern \"C\" int proj_number() { return 7; }\n"
MODULE = "extern \"C\" int proj_number();\nextern \"C\" int twice() { return 2 * proj_number(); }\n"


@pytest.fixture
def b(tmp_path, monkeypatch):
    from hidden_state_projection_gb300 import build as m
    try:
        m._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    if m._py_missing() is not None:
        pytest.skip("no headers for the Python module")
    csrc, lib = tmp_path / "csrc", tmp_path / "_lib"
    csrc.mkdir()
    (csrc / "one.cu").write_text(LIBRARY)
    (csrc / "py_cache.cpp").write_text(MODULE)
    monkeypatch.delenv("CXX", raising=False)
    for name, value in (("CSRC", csrc), ("LIB_DIR", lib), ("OBJ_DIR", lib / "obj"), ("LIB_PATH", lib / "libhsp_proj.so"),
                        ("PY_SRC", csrc / "py_cache.cpp"), ("PY_PATH", lib / "hsp_cache_py.so")):
        monkeypatch.setattr(m, name, str(value))
    return m


def times(b):
    return [os.stat(p).st_mtime_ns for p in (b.LIB_PATH, b.PY_PATH, os.path.join(b.OBJ_DIR, "py_cache.o"))]


@pytest.mark.parametrize("missing", ["torch", "python", "compiler"])
def test_library_without_the_python_module(b, monkeypatch, capsys, missing):
    """A C user's machine: no torch, no Python headers, or no C++ compiler by that name."""
    if missing == "torch":
        monkeypatch.setattr(b, "_torch_dir", lambda: None)
    elif missing == "python":
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
    else:
        monkeypatch.setattr(b, "_cxx", lambda: None)
    assert b.build() == b.LIB_PATH
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.PY_PATH)
    assert "hsp_cache_py.so is not built" in capsys.readouterr().err


def test_library_is_linked_before_a_broken_module_is_reported(b):
    with open(b.PY_SRC, "a") as f:
        f.write("#error broken\n")
    for _ in range(2):                                      # and again: a failed object is not taken for a made one
        with pytest.raises(RuntimeError, match="broken"):
            b.build()
        assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.PY_PATH)


def test_a_broken_kernel_is_reported(b):
    with open(os.path.join(b.CSRC, "one.cu"), "a") as f:
        f.write("#error broken\n")
    with pytest.raises(RuntimeError, match="broken"):
        b.build()
    assert not os.path.exists(b.LIB_PATH)


def test_module_is_made_anew_for_another_torch(b, monkeypatch, tmp_path):
    b.build()
    first = times(b)
    b.build()
    assert times(b) == first                                # nothing to do
    other = tmp_path / "torch"
    for d in ("include", "lib"):
        os.makedirs(other / d)
    os.symlink(os.path.join(b._torch_dir(), "include", "ATen"), other / "include" / "ATen")
    for f in os.listdir(os.path.join(b._torch_dir(), "lib")):
        os.symlink(os.path.join(b._torch_dir(), "lib", f), other / "lib" / f)
    (other / "version.py").write_text("__version__ = '99'\n")
    monkeypatch.setattr(b, "_torch_dir", lambda: str(other))
    b.build()
    second = times(b)
    assert second[0] == first[0] and second[1] > first[1] and second[2] > first[2]
    (other / "version.py").write_text("__version__ = '100'\n")   # another version in the same place
    b.build()
    third = times(b)
    assert third[0] == first[0] and third[2] > second[2]


def test_a_compiler_of_several_words(b, monkeypatch):
    env = shutil.which("env")
    monkeypatch.setenv("CXX", f"{env} g++")
    b.build()
    assert os.path.exists(b.PY_PATH)
    code = f"import ctypes; ctypes.CDLL({b.LIB_PATH!r}); print(ctypes.CDLL({b.PY_PATH!r}).twice())"
    r = subprocess.run([sys.executable, "-c", "import torch; " + code], capture_output=True, text=True)
    assert r.stdout.strip() == "14", r.stderr
