"""Build libsparsepr.so (sm_100a) in-tree with nvcc, and the extension module _marshal with g++.

    python -m free_block_sparse_means_b200.build [--force] [--verbose]

Objects go to _build/ at the repository root; the shared library goes to
free_block_sparse_means_b200/lib/.  Rebuilds only when a source is newer than
the library.  _marshal (the operators' calls from Python, against the installed
torch's headers, under a name that tells both) goes beside it.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys

from ._binding import MARSHAL_PATH

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libsparsepr.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL = MARSHAL_PATH
BUILD = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in sources() + headers() + [__file__])


def marshal_command():
    """The g++ command of _marshal; the process that loads it has torch's libraries already."""
    import sysconfig

    import torch
    headers = os.path.join(os.path.dirname(torch.__file__), "include")
    inc = [headers, os.path.join(headers, "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], INCLUDE,
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[a for i in inc for a in ("-isystem", i)], MARSHAL_SRC, "-o", MARSHAL + ".tmp",
            "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def marshal_up_to_date() -> bool:
    return os.path.exists(MARSHAL) and all(
        os.path.getmtime(f) <= os.path.getmtime(MARSHAL)
        for f in [MARSHAL_SRC, os.path.join(INCLUDE, "sparsepr.h"), __file__])


def build(force: bool = False, verbose: bool = False) -> str:
    extension = None
    os.makedirs(LIBDIR, exist_ok=True)
    if force or not marshal_up_to_date():
        extension = subprocess.Popen(marshal_command(), stdout=subprocess.PIPE,
                                     stderr=subprocess.STDOUT, text=True)
    try:
        if force or not up_to_date():
            build_library(verbose)
    finally:
        if extension:
            out, _ = extension.communicate()
            if extension.returncode == 0:
                os.replace(MARSHAL + ".tmp", MARSHAL)
            else:
                sys.stderr.write(out)
    if extension and extension.returncode:
        raise RuntimeError("g++ failed for: " + MARSHAL_SRC)
    return LIB


def build_library(verbose: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    procs, objs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [cc, *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            sys.stderr.write(out)
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB + ".tmp"
    subprocess.check_call([cc, *ARCH, "-shared", "--cudart=static", "-o", tmp, *objs])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
