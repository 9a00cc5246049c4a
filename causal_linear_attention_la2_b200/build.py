"""Builds libla2.so in-tree with nvcc for sm_100a.

    python -m causal_linear_attention_la2_b200.build [--verbose-ptxas] [--force]

The library has two translation units that include their kernels:
csrc/la2_api.cu (linear attention with a decay) and csrc/gdr_api.cu (the gated
delta rule and the state pool).  They are compiled side by side into _build/,
each only when one of its sources is newer.  cudart is linked statically; the
CUDA driver is reached through cudaGetDriverEntryPoint, so the library links no
libcuda.
"""
from __future__ import annotations

import argparse
import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libla2.so")
OBJ = os.path.join(PKG, "_build")
UNITS = ("la2_api.cu", "gdr_api.cu")

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  [os.path.join(INCLUDE, "la2.h")])


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def unit_sources(unit: str) -> list[str]:
    """A translation unit, what it includes (transitively) and this file."""
    seen, todo = [], [os.path.join(CSRC, unit)]
    while todo:
        path = todo.pop()
        if path in seen:
            continue
        seen.append(path)
        with open(path) as f:
            names = re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M)
        todo += [p for n in names for p in (os.path.join(CSRC, n), os.path.join(INCLUDE, n))
                 if os.path.exists(p)]
    return seen + [os.path.abspath(__file__)]


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not verbose_ptxas and not needs_build():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    flags = [*ARCH_FLAGS, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        flags.append("-Xptxas=-v")
    objs, jobs = [], []
    for unit in UNITS:
        obj = os.path.join(OBJ, unit + ".o")
        objs.append(obj)
        old = not os.path.exists(obj) or any(os.path.getmtime(p) > os.path.getmtime(obj)
                                             for p in unit_sources(unit))
        if force or verbose_ptxas or old:
            tmp = obj + f".tmp{os.getpid()}"
            cmd = [nvcc_path(), *flags, "-c", "-o", tmp, os.path.join(CSRC, unit)]
            jobs.append((cmd, subprocess.Popen(cmd), tmp, obj))
    failed = [cmd for cmd, p, _, _ in jobs if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, _, tmp, obj in jobs:
        os.replace(tmp, obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc_path(), *ARCH_FLAGS, "-Xcompiler", "-fPIC", "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
    return 0


if __name__ == "__main__":
    sys.exit(main())
