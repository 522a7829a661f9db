"""Build the CUDA library libhsp_proj.so in-tree (sm_103a only).

Every translation unit under csrc/ is compiled in parallel with
``nvcc -gencode arch=compute_103a,code=sm_103a`` and linked into
``_lib/libhsp_proj.so``.  No cmake, no torch extension machinery.
``csrc/py_cache.cpp``, the tensor side of the paged cache's calls, is compiled by the
host compiler against torch's headers and linked to that library as
``_lib/hsp_cache_py.so``.
"""
from __future__ import annotations

import glob
import importlib.util
import os
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


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch not found: its headers are needed for the Python side")
    return list(spec.submodule_search_locations)[0]


def _py_compile(obj: str):
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler: the Python side cannot be built")
    inc = os.path.join(_torch_dir(), "include")
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", f"-I{INCLUDE}", "-isystem", inc, "-isystem",
            os.path.join(inc, "torch", "csrc", "api", "include"), f"-I{sysconfig.get_paths()['include']}", "-c", PY_SRC, "-o", obj]


def _py_link(obj: str, out: str):
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    return [cxx, "-shared", "-o", out, obj, f"-L{os.path.join(_torch_dir(), 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10",
            f"-L{LIB_DIR}", "-l:libhsp_proj.so", "-Wl,-rpath,$ORIGIN"]


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
    py_obj = os.path.join(OBJ_DIR, "py_cache.o")
    if force or _stale(py_obj, [PY_SRC, os.path.join(INCLUDE, "proj.h")]):
        cmd = _py_compile(py_obj)
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((PY_SRC, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out))
        elif out and (verbose or ptxas_info):
            print(out, end="")
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
