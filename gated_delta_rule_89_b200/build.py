"""Build libgdr.so in-tree with nvcc for sm_100a (B200).

    python -m gated_delta_rule_89_b200.build

compiles every ``csrc/*.cu`` (in parallel, into objects under ``_build/``; only
what changed) and links them into one shared library next to this file.  The
CUDA runtime is linked statically, so the library runs beside any PyTorch
build; the driver API (tensor maps) is reached through the runtime's entry
point query, so no link against libcuda is needed.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libgdr.so")
OBJ = os.path.join(PKG, "_build")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(PKG, "csrc", "*.cuh"))) + \
        [os.path.join(ROOT, "include", "gdr.h")]


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in deps())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not needs_build():
        return LIB
    # objects made with other flags lie in a folder of their own: no later build links them
    objdir = os.path.join(OBJ, "extra") if extra else OBJ
    os.makedirs(objdir, exist_ok=True)
    headers = [p for p in deps() if not p.endswith(".cu")] + [os.path.abspath(__file__)]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        if not force and not extra and os.path.exists(obj) and \
                all(os.path.getmtime(obj) >= os.path.getmtime(p) for p in [src, *headers]):
            return obj
        run([nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "--expt-relaxed-constexpr",
             "-Xcompiler", "-fPIC,-fvisibility=hidden",
             "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc"),
             *extra, "-c", "-o", obj + ".tmp", src])
        os.replace(obj + ".tmp", obj)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
        objects = list(pool.map(compile_one, sources()))
    run([nvcc(), *ARCH, "-Xcompiler", "-fPIC", "-shared", "-o", LIB + ".tmp", *objects])
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
