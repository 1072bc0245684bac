"""Builds libgdn.so in-tree from csrc/*.cu for sm_103a with nvcc.

Each translation unit compiles in parallel to an object file, then nvcc links
the shared library into ``_build/libgdn.so``.  ``_build/_front.*.so`` is the
binding's way into the layer operators, host code over torch's C++ headers, and
belongs to one version of torch and Python, which its name holds.  Rebuilds only
what is stale.
Usage: ``python -m gated_delta_rule_47_gb300.build [--force]``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libgdn.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn.so")


def _deps():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target, sources):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def _compile(src, extra):
    obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
    if _stale(obj, [src] + _deps()):
        cmd = [nvcc()] + ARCH + FLAGS + extra + ["-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def front_path(torch_version: str) -> str:
    """The front's file for this Python and a version of torch: it is built against
    the C++ interfaces of both, which have no stable ABI."""
    return os.path.join(OUT_DIR, f"_front.{sys.implementation.cache_tag}-torch{torch_version}.so")


def _front():
    src = os.path.join(CSRC, "front.cpp")
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    # torch.__version__, without the time that importing torch takes
    front = front_path(str(runpy.run_path(os.path.join(torch, "version.py"))["__version__"]))
    if _stale(front, [src, os.path.join(INCLUDE, "gdn.h")]):
        tmp = front + f".{os.getpid()}.tmp"
        includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(torch, "include"),
                    os.path.join(torch, "include", "torch", "csrc", "api", "include")]
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", *(f"-I{d}" for d in includes), src,
               "-o", tmp, "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed for {src}:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, front)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for f in glob.glob(os.path.join(OUT_DIR, "*.o")) + glob.glob(os.path.join(OUT_DIR, "_front.*so")):
            os.remove(f)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        front = ex.submit(_front)
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
        front.result()
    if force or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
