"""Build step: compile the CUDA sources of the package into lib/libpack3d.so for sm_100a, then the
binding's helper for lists of tensors into lib/ (tensor_list_path). The library needs nvcc alone; where
the helper cannot be built, that is a warning, and the calls over lists of tensors say so when used.

Usage: python -m geometry_aware_local_pack3d_b200.build [--force] [--verbose]
Objects go to _build/ (git-ignored); the shared library is written in-tree so it travels
with the source tree.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "lib", "libpack3d.so")
LIST_SRC = os.path.join(CSRC, "tensor_list.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O3",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _compile(src, verbose, extra):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    return obj, r.stderr


def tensor_list_path():
    """The helper's file: it is compiled against torch's classes and Python's ABI, so both versions
    are in its name, and one that was built for others is not found."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    key = f"torch{torch.__version__}-cxx{abi}-{sysconfig.get_config_var('SOABI')}"
    return os.path.join(PKG, "lib", f"_tensor_list-{key}.so")


def build_tensor_list(force=False):
    """The host helper that reads a list of tensors (a CPython module over torch's headers)."""
    out = tensor_list_path()
    newest = max(os.path.getmtime(LIST_SRC), os.path.getmtime(__file__))
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest:
        return out
    import torch
    os.makedirs(os.path.dirname(out), exist_ok=True)
    root = os.path.dirname(torch.__file__)
    tmp = out + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], LIST_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {LIST_SRC}:\n{r.stderr}")
    os.replace(tmp, out)
    return out


def build(force=False, verbose=False, extra=()):
    lib = build_library(force, verbose, extra)
    try:
        build_tensor_list(force)
    except (RuntimeError, OSError, ImportError) as e:
        warnings.warn(f"the helper for lists of tensors was not built: {e}")
    return lib


def build_library(force=False, verbose=False, extra=()):
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    srcs = sources()
    newest = max(os.path.getmtime(p) for p in srcs + headers() + [__file__])
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose, list(extra)), srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
