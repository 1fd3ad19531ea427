"""Build libkmeans_b200.so in-tree with nvcc for sm_100a.

Usage: python -m exact_lloyd_means_assign_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkmeans_b200.so")
# translation units: the k-means library proper, then one per operator family
UNITS = ["km_lib.cu", "km_lookup.cu", "km_matvec4.cu", "km_xent.cu"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc():
    cand = [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh", ".h"))] + [
        os.path.join(INCLUDE, "kmeans_b200.h")]


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in _sources())


def _unit_sources(unit):
    """The files a unit is compiled from: itself and, transitively, the local headers it includes."""
    seen, todo = set(), [os.path.join(CSRC, unit)]
    while todo:
        path = todo.pop()
        if path in seen:
            continue
        seen.add(path)
        with open(path) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M):
                for d in (CSRC, INCLUDE):
                    if os.path.exists(os.path.join(d, name)):
                        todo.append(os.path.join(d, name))
    return seen


def build(force=False, verbose=False):
    """Compile the CUDA library (its units side by side) unless it is up to date."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs, running = [], []
    for unit in UNITS:
        obj = os.path.join(objdir, unit[:-3] + ".o")
        objs.append(obj)
        if not force and os.path.exists(obj) and \
                all(os.path.getmtime(s) <= os.path.getmtime(obj) for s in _unit_sources(unit)):
            continue
        cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
               "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
               "-c", os.path.join(CSRC, unit), "-o", obj + ".tmp"]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd))
        running.append((obj, cmd, subprocess.Popen(cmd)))
    failed = None
    for obj, cmd, p in running:
        if p.wait() != 0:
            failed = cmd
        else:
            os.replace(obj + ".tmp", obj)
    if failed:
        raise subprocess.CalledProcessError(1, failed)
    subprocess.run([nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", LIB + ".tmp", *objs], check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
