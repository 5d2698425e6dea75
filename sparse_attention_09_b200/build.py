"""Builds libdsa.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a, and _marshal.so (the Python
module that checks tensors and calls it) with g++.

Usage: python sparse_attention_09_b200/build.py [--verbose]
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_PATH = os.path.join(PKG_DIR, "libdsa.so")
MARSHAL_PATH = os.path.join(PKG_DIR, "_marshal.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def sources():
    return [os.path.join(CSRC, "dsa_api.cu")]


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "marshal.cpp"] + [os.path.join(ROOT, "include", "dsa.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def marshal_target() -> str:
    """What _marshal.so depends on beside its sources: the torch whose objects it reads, Python's and C++'s binary interface.
    It is written into the module when it is compiled."""
    import sysconfig

    import torch

    return f"dsa_marshal for torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}, cxx11 abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)};"


def marshal_current() -> bool:
    """Whether _marshal.so exists and was compiled for this torch and Python."""
    if not os.path.exists(MARSHAL_PATH):
        return False
    with open(MARSHAL_PATH, "rb") as f:
        return marshal_target().encode() in f.read()


def _build_marshal(force: bool) -> None:
    """Compile _marshal.so against the libraries that torch loads (found by their names: torch is imported first)."""
    src = os.path.join(CSRC, "marshal.cpp")
    deps = [src, os.path.join(ROOT, "include", "dsa.h")]
    if not force and marshal_current() and all(os.path.getmtime(d) <= os.path.getmtime(MARSHAL_PATH) for d in deps):
        return
    import sysconfig

    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = MARSHAL_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DDSA_MARSHAL_TARGET="{marshal_target()}"',
           "-isystem", os.path.join(base, "include"), "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"), src, "-o", tmp,
           "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           "-L", PKG_DIR, "-ldsa", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, cwd=ROOT, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, MARSHAL_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library and the Python module if a source is newer than what is built; returns the library's path."""
    _build_library(force, verbose)
    _build_marshal(force)
    return LIB_PATH


def _build_library(force: bool, verbose: bool) -> None:
    if not force and not _stale():
        return
    tmp = LIB_PATH + ".tmp"
    cmd = [_nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), *sources(), "-o", tmp]
    if verbose:
        cmd += ["-Xptxas", "-v"]
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, cwd=ROOT, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stdout + res.stderr)
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB_PATH)
