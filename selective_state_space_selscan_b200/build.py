"""Build libselscan.so in-tree with nvcc for sm_100a.

The shared library is the product: it exports the C ABI declared in
include/selscan.h.  Python reaches it through ctypes (see __init__.py).
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libselscan.so")
SOURCES = [os.path.join(CSRC, f) for f in ("selscan_api.cu", "layer_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cuh", ".h"))] + [
    os.path.join(ROOT, "include", f) for f in os.listdir(os.path.join(ROOT, "include"))
    if f.endswith(".h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
    "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile libselscan.so unless it is newer than every source."""
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(p) for p in DEPS)):
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    flags = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    objs = [f"{tmp}.{i}.o" for i in range(len(SOURCES))]
    cmds = [[*flags, *extra, "-c", "-o", o, src] for o, src in zip(objs, SOURCES)]
    try:
        jobs = []
        for cmd in cmds:  # one compiler per source, side by side
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            jobs.append(subprocess.Popen(cmd))
        for cmd, rc in [(cmd, job.wait()) for cmd, job in zip(cmds, jobs)]:
            if rc:
                raise subprocess.CalledProcessError(rc, cmd)
        subprocess.check_call([*flags, "-shared", "-o", tmp, *objs, "-lcuda"])
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
