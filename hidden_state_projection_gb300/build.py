"""Build the CUDA library libhsp_proj.so in-tree (sm_103a only).

Every translation unit under csrc/ is compiled in parallel with
``nvcc -gencode arch=compute_103a,code=sm_103a`` and linked into
``_lib/libhsp_proj.so``.  No cmake, no torch extension machinery.
``csrc/py_cache.cpp``, the tensor side of the paged cache's calls, is compiled by the
host compiler against torch's headers and linked to that library as
``_lib/hsp_cache_py.so``.  The library needs neither Python's nor torch's headers: it is
linked first, and without them (a C user's machine) the Python module is left out.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shlex
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(HERE, "_lib")
OBJ_DIR = os.path.join(LIB_DIR, "obj")
LIB_PATH = os.path.join(LIB_DIR, "libhsp_proj.so")
PY_SRC = os.path.join(CSRC, "py_cache.cpp")
PY_PATH = os.path.join(LIB_DIR, "hsp_cache_py.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir():
    """torch's package folder, or None."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec is not None and spec.submodule_search_locations else None


def _cxx():
    """The C++ compiler's words (CXX may have several), or None."""
    words = shlex.split(os.environ.get("CXX", "")) or [shutil.which("g++") or shutil.which("c++") or ""]
    return words if words[0] else None


def _py_missing():
    """What the Python module cannot be built without and is not here, or None."""
    if _cxx() is None:
        return "C++ compiler"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    if _torch_dir() is None or not os.path.exists(os.path.join(_torch_dir(), "include", "ATen", "ATen.h")):
        return "torch's headers"
    return None


def _py_compile(obj: str):
    inc = os.path.join(_torch_dir(), "include")
    return [*_cxx(), "-O2", "-std=c++17", "-fPIC", "-Wall", f"-I{INCLUDE}", "-isystem", inc, "-isystem",
            os.path.join(inc, "torch", "csrc", "api", "include"), f"-I{sysconfig.get_paths()['include']}", "-c", PY_SRC, "-o", obj]


def _py_link(obj: str, out: str):
    return [*_cxx(), "-shared", "-o", out, obj, f"-L{os.path.join(_torch_dir(), 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10",
            f"-L{LIB_DIR}", "-l:libhsp_proj.so", "-Wl,-rpath,$ORIGIN"]


def _py_made_with(cmd) -> str:
    """What the object depends on besides its sources: the command, Python and torch, whose C++ types it uses."""
    version = os.path.join(_torch_dir(), "version.py")
    torch_is = open(version).read() if os.path.exists(version) else ""
    return "\n".join([shlex.join(cmd), sys.version, torch_is])


def _read(path: str) -> str:
    return open(path).read() if os.path.exists(path) else ""


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc = _nvcc()
    headers = _headers()
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc, *ARCH, *CFLAGS, "-c", src, "-o", obj]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                                text=True)))
    py_obj, py_stamp = os.path.join(OBJ_DIR, "py_cache.o"), os.path.join(OBJ_DIR, "py_cache.made_with")
    missing, py_proc, py_out = _py_missing(), None, ""
    if missing is None:
        cmd = _py_compile(py_obj)
        made_with = _py_made_with(cmd)
        if force or _stale(py_obj, [PY_SRC, os.path.join(INCLUDE, "proj.h")]) or _read(py_stamp) != made_with:
            if verbose:
                print(" ".join(cmd), flush=True)
            if os.path.exists(py_stamp):
                os.remove(py_stamp)
            py_proc = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out))
        elif out and (verbose or ptxas_info):
            print(out, end="")
    if py_proc is not None:
        py_out, _ = py_proc.communicate()
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"compilation failed:\n{msg}")
    if force or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB_PATH)
    if missing is not None:
        print(f"{PY_PATH} is not built ({missing} not found): "
              "the paged cache's Python calls need it, the C library does not", file=sys.stderr, flush=True)
        return LIB_PATH
    if py_proc is not None:
        if py_proc.returncode != 0:
            raise RuntimeError(f"{LIB_PATH} is built, but not the Python module:\n--- {PY_SRC}\n{py_out}")
        if py_out and verbose:
            print(py_out, end="")
        with open(py_stamp, "w") as f:
            f.write(made_with)
    if force or _stale(PY_PATH, [py_obj, LIB_PATH]):
        tmp = PY_PATH + f".tmp{os.getpid()}"
        cmd = _py_link(py_obj, tmp)
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, PY_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
