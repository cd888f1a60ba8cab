"""Build ``libgdr.so`` (the C-ABI library) in-tree with nvcc for sm_100a, and
the compiled torch front end of some of its entry points (``_gdr_torch*.so``,
named after the torch and Python it is for).

Usage: ``python -m gated_delta_rule_93_b200.build [--force] [-v]``.
Each ``csrc/*.cu`` compiles to ``_build/*.o`` in parallel (skipped when the
object is newer than its inputs), then nvcc links the shared library with
the CUDA runtime linked statically, so the library loads on a machine with
no GPU driver (only the first CUDA call needs one).  The front end is host
code, compiled with g++ against the installed torch; where that fails the
library is built all the same, with a warning, and the entry points behind the
front end raise.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import warnings

from .binding import NATIVE_PATH as NATIVE

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgdr.so")
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE,
                 "-I" + CSRC, "--expt-relaxed-constexpr"]


def _deps():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target, inputs):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in inputs)


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC] + CFLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    return obj, r.stderr


def _compile_native(src):
    """The torch front end: g++, linked to the installed torch."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(NVCC))
    inc = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths(),
           os.path.join(cuda, "include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = NATIVE + ".tmp%d" % os.getpid()
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{p}" for p in inc), src, "-o", tmp, "-L" + libs, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed for {src}:\n{r.stderr}")
    os.replace(tmp, NATIVE)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = _deps()
    todo = [s for s in srcs
            if force or _stale(os.path.join(BUILD, os.path.basename(s)[:-3] + ".o"), [s] + deps)]
    logs = []
    front = os.path.join(CSRC, "gdr_torch.cpp")
    front_stale = force or _stale(NATIVE, [front] + glob.glob(os.path.join(INCLUDE, "*.h")))
    front_done = None
    if todo or front_stale:
        workers = max(1, min(len(todo) + 1, os.cpu_count() or 1))
        with cf.ThreadPoolExecutor(max_workers=workers) as ex:
            if front_stale:
                front_done = ex.submit(_compile_native, front)
            for obj, log in ex.map(lambda s: _compile(s, verbose), todo):
                logs.append(log)
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if force or todo or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [NVCC] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc link failed:\n" + r.stderr)
        os.replace(tmp, LIB)
    failure = front_done.exception() if front_done else None
    if failure:
        if os.path.exists(NATIVE):
            os.unlink(NATIVE)  # of an older source
        warnings.warn(f"{LIB} is built, its compiled torch front end is not: {failure}",
                      RuntimeWarning, stacklevel=2)
    if verbose:
        sys.stderr.write("".join(logs))
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(a.force, a.verbose))


if __name__ == "__main__":
    main()
