"""Compile the CUDA verify library (sm_103a) into the package directory.

One -gencode; the translation units are compiled in parallel and linked into
one library.  nvcc cross-compiles without a GPU and builds natively on the GPU
host in well under a minute.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libspec_verify.so")
SOURCES = [os.path.join(PKG, "csrc", n + ".cu")
           for n in ("spec_verify", "probs", "kv_append", "attention")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA verify library cannot be built")
    return path


def inputs() -> list[str]:
    return SOURCES + glob.glob(os.path.join(PKG, "csrc", "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libspec_verify.so if it is missing or older than its sources."""
    if not (force or stale()):
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    base = [nvcc(), "-O3", *ARCH, "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]
    if verbose:
        base.insert(1, "-Xptxas=-v")
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.basename(src) + ".o") for src in SOURCES]
        runs = [subprocess.Popen([*base, "-c", "-o", obj, src]) for src, obj in zip(SOURCES, objs)]
        codes = [r.wait() for r in runs]
        if any(codes):
            raise RuntimeError(f"nvcc failed on {[s for s, c in zip(SOURCES, codes) if c]}")
        subprocess.run([*base, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
