"""Build libsparsepool.so in-tree from csrc/*.cu for sm_103a (GB300).

Each translation unit is compiled by nvcc in parallel, then linked into
``block_sparse_long_pool_gb300/libsparsepool.so``.  No cmake, no torch extension
machinery: the product is a plain C-ABI shared library.  ``_marshal_<torch version>.so`` beside
it, from csrc/marshal.cpp by g++, passes tensors from Python to three of its calls; it is left
out where there is no torch, which the library does not need.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsparsepool.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def flags(extra=()) -> list[str]:
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                   f"-I{INCLUDE}", f"-I{CSRC}", "--expt-relaxed-constexpr"] + list(extra)


def _stale(obj: str, src: str, deps: list[str]) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(x) > t for x in [src] + deps)


def build_marshal(verbose: bool = False, force: bool = False) -> str:
    import torch
    out = os.path.join(PKG, f"_marshal_{torch.__version__}.so")   # reads that version's tensor objects
    src = os.path.join(CSRC, "marshal.cpp")
    if force or _stale(out, src, [os.path.join(INCLUDE, "sparse_pool.h"), os.path.abspath(__file__)]):
        tmp = out + f".{os.getpid()}.tmp"
        root = os.path.dirname(torch.__file__)
        cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-Wall", "-std=c++17", "-shared", "-fPIC",
               "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
               *(f"-isystem{x}" for x in (f"{root}/include", f"{root}/include/torch/csrc/api/include",
                                          sysconfig.get_paths()["include"])),
               src, f"-L{root}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("g++ failed on marshal.cpp")
        os.replace(tmp, out)
    return out


def build(verbose: bool = False, extra=(), force: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(INCLUDE, "sparse_pool.h"),
                                                             os.path.abspath(__file__)]
    cc = nvcc()
    jobs = []
    objs = []
    for src in srcs:
        obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, src, deps):
            jobs.append([cc] + flags(extra) + ["-c", src, "-o", obj])
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        marshal = ex.submit(build_marshal, verbose, force) if importlib.util.find_spec("torch") else None
        results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
    for cmd, r in zip(jobs, results):
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {cmd[-3]}")
    if force or jobs or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [cc] + ARCH + ["-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, LIB)
    if marshal is not None:
        marshal.result()
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
