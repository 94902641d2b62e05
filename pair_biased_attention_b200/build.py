"""Builds libpba.so (the C-ABI library) in-tree for sm_100a with nvcc.

    python -m pair_biased_attention_b200.build [--verbose]

Every csrc/*.cu is compiled on its own, all of them at once, and linked
against the static CUDA runtime, so the library carries no dependency on the
runtime that PyTorch loads.  Rebuilds only when a source or the header is newer
than the .so.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libpba.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-cudart", "static",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpba.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  [os.path.join(INCLUDE, "pba.h")])


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    cmd = [_nvcc(), *NVCC_FLAGS]
    with tempfile.TemporaryDirectory(dir=PKG, prefix="_build_") as tmp:
        objects, running = [], []
        for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
            objects.append(os.path.join(tmp, os.path.basename(src) + ".o"))
            running.append(subprocess.Popen(cmd + (["-Xptxas", "-v"] if verbose else []) +
                                            ["-I", INCLUDE, "-I", CSRC, "-c", "-o", objects[-1], src]))
        # every compiler is waited for before the folder goes, also when one has failed
        if any([p.wait() for p in running]):
            raise RuntimeError("nvcc failed")
        subprocess.check_call([*cmd, "-shared", "-o", LIB + ".tmp", *objects])
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv or "--verbose" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
