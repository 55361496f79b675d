"""Builds libprox.so (all CUDA sources, sm_100a) and the Python entry of the
4-bit operators (_decode4.so) next to this file.

Usage: python activation_sparse_swiglu_b200/build.py [--force] [--verbose] [--ptxas-info]
(run by path: importing the package loads libprox.so, which may be missing or stale)
"""

from __future__ import annotations

import argparse
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libprox.so")
ENTRY = os.path.join(PKG, "_decode4.so")
ENTRY_SOURCE = os.path.join(CSRC, "decode4_py.cpp")

SOURCES = ["prox_api.cu", "token.cu", "batch.cu", "pack.cu", "calibrate.cu", "misc.cu",
           "decode4_api.cu", "linear4.cu", "kv4.cu", "attend4.cu", "pages.cu"]
HEADERS = ["prox_device.cuh", "prox_internal.h", "select.cuh", "token_args.cuh", "stage1.cuh",
           "stage2.cuh", "api_util.h", "decode4.h", "quant4.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libprox.so")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(INCLUDE, "prox.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not ptxas_info and up_to_date():
        build_entry()
        return LIB
    nvcc = _nvcc()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-shared", "-o", tmp]
    if ptxas_info:
        cmd += ["-Xptxas", "-v"]
    cmd += [os.path.join(CSRC, s) for s in SOURCES]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"nvcc failed ({proc.returncode}):\n{proc.stdout}\n{proc.stderr}")
    if ptxas_info or verbose:
        sys.stderr.write(proc.stderr)
    os.replace(tmp, LIB)
    build_entry(force=force, verbose=verbose)
    return LIB


def _torch_dir() -> str:
    import importlib.util
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def entry_tag() -> str:
    """What _decode4.so is compiled against: its C++ interface is that of one
    torch and one Python."""
    with open(os.path.join(_torch_dir(), "version.py")) as fh:
        version = re.search(r"^__version__ = '([^']*)'", fh.read(), re.M).group(1)
    return f"torch {version}, {sys.implementation.cache_tag}"


def entry_up_to_date() -> bool:
    inputs = [ENTRY_SOURCE, os.path.join(INCLUDE, "prox.h"), os.path.abspath(__file__)]
    if not os.path.exists(ENTRY) or any(os.path.getmtime(f) > os.path.getmtime(ENTRY) for f in inputs):
        return False
    with open(ENTRY, "rb") as fh:
        return entry_tag().encode() + b"\0" in fh.read()


def build_entry(force: bool = False, verbose: bool = False) -> str:
    """_decode4.so: a CPython module over torch's tensors and libprox.so."""
    if not force and entry_up_to_date():
        return ENTRY
    import sysconfig
    torch_dir = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = ENTRY + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-o", tmp, ENTRY_SOURCE,
           f'-DPROX_BUILT_FOR="{entry_tag()}"', "-I", INCLUDE, "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           "-L", PKG, "-l:libprox.so", "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"g++ failed ({proc.returncode}):\n{proc.stdout}\n{proc.stderr}")
    os.replace(tmp, ENTRY)
    return ENTRY


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose, ptxas_info=args.ptxas_info))
