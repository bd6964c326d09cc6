"""Build libselscan.so in-tree with nvcc for sm_100a.

The shared library is the product: it exports the C ABI declared in
include/selscan.h.  Python reaches it through ctypes (see __init__.py).
"""
from __future__ import annotations

import os
import subprocess
import sys

from . import BIND_PATH as BIND
from . import bind_fits, bind_stamp

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libselscan.so")
SOURCES = [os.path.join(CSRC, f) for f in ("selscan_api.cu", "layer_api.cu")]
BIND_SRC = os.path.join(CSRC, "bind.cpp")
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


def bind_headers() -> list[str]:
    """Directories of the headers that csrc/bind.cpp needs, or none where torch's
    or Python's are not installed."""
    import importlib.util
    import sysconfig

    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return []
    base = os.path.join(spec.submodule_search_locations[0], "include")
    dirs = [base, os.path.join(base, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"]]
    wanted = (os.path.join(base, "torch", "csrc", "autograd", "python_variable.h"),
              os.path.join(dirs[2], "Python.h"))
    return dirs if all(os.path.exists(p) for p in wanted) else []


def build_bind(force: bool = False, verbose: bool = False) -> str | None:
    """Compile _bind.so (tensors to the C ABI, csrc/bind.cpp) against the
    installed torch, unless it was built for that and is newer than its sources.
    None, with a note, where torch's or Python's headers are not installed: every
    call then goes through ctypes, which needs none."""
    dirs = bind_headers()
    if not dirs:
        print("no headers of torch or Python here: _bind.so is not built, calls go through ctypes",
              file=sys.stderr)
        return None
    header = os.path.join(ROOT, "include", "selscan.h")
    if (not force and bind_fits(BIND)
            and os.path.getmtime(BIND) >= max(os.path.getmtime(p) for p in (BIND_SRC, header))):
        return BIND
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(ROOT, "include"), *dirs,
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden", f'-DSELSCAN_BIND_STAMP="{bind_stamp()}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{p}" for p in inc], "-o", tmp, BIND_SRC, "-L", PKG, "-l:libselscan.so",
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, BIND)
    return BIND


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    build_bind(force="--force" in sys.argv, verbose=True)
