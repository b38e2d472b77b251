"""Builds libblk.so (the C-ABI library) in-tree for sm_103a with nvcc, and _fastcall.so.

Each .cu translation unit compiles in parallel to an object under _build/, then
nvcc links the shared library next to this file. A unit is recompiled only when
it, or a header it includes, is newer than its object. _fastcall.so, the compiled
argument handling of the packed calls (csrc/fastcall.cpp), is built beside it
against the installed torch.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libblk.so")
FAST_SRC = os.path.join(CSRC, "fastcall.cpp")
FAST_OBJ = os.path.join(BUILD, "fastcall.o")
FAST = os.path.join(HERE, "_fastcall.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-I", os.path.join(ROOT, "include")]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(src, obj, headers):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(f) > t for f in [src, *headers])


def _fastcall_for() -> str:
    """What _fastcall.so's binary interface depends on; _build/fastcall.for says what it was built for."""
    import torch

    return f"torch {torch.__version__} in {os.path.dirname(torch.__file__)}, C++11 ABI " \
           f"{int(torch._C._GLIBCXX_USE_CXX11_ABI)}, python {sysconfig.get_config_var('EXT_SUFFIX')}"


def _built_for() -> str | None:
    try:
        with open(os.path.join(BUILD, "fastcall.for")) as f:
            return f.read()
    except OSError:
        return None


def _cuda_include() -> str:
    nvcc = _nvcc()
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(nvcc) or nvcc))), "include")


def _compile_fastcall() -> subprocess.Popen | None:
    """Starts the compiler on fastcall.cpp if its object is older than its sources, or made for another
    torch or Python."""
    import torch

    if _built_for() == _fastcall_for() and not _stale(FAST_SRC, FAST_OBJ, glob.glob(os.path.join(ROOT, "include", "*.h"))):
        return None
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-I", root, "-I", os.path.join(root, "torch", "csrc", "api", "include"),
           "-I", _cuda_include(), "-c", FAST_SRC, "-o", FAST_OBJ]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _link_fastcall():
    """Links _fastcall.so against the libblk.so beside it and the installed torch."""
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-shared", FAST_OBJ, "-o", FAST, "-L", HERE, "-l:libblk.so", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda",
           "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")


def build(verbose: bool = False, jobs: int | None = None) -> str:
    """Compiles the CUDA sources and links libblk.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    fast = _compile_fastcall()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    todo = [(s, o) for s, o in zip(srcs, objs) if _stale(s, o, headers)]

    def compile_one(so):
        s, o = so
        cmd = [nvcc, *ARCH, *FLAGS, "-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(s)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return o

    if todo:
        with ThreadPoolExecutor(max_workers=jobs or min(len(todo), os.cpu_count() or 4)) as ex:
            list(ex.map(compile_one, todo))
    if todo or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    if fast is not None:
        out, _ = fast.communicate()
        if fast.returncode != 0:
            raise RuntimeError(f"g++ failed on {os.path.basename(FAST_SRC)}:\n{out}")
    if fast is not None or _stale(FAST_OBJ, FAST, []):
        _link_fastcall()
    if fast is not None:
        with open(os.path.join(BUILD, "fastcall.for"), "w") as f:
            f.write(_fastcall_for())
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
