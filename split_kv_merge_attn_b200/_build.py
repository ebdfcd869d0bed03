"""Builds the in-tree shared library ``libsplitkv.so`` for sm_100a with nvcc, and
``_skv_torch.<PyTorch>.<Python>.so``, the extension module that marshals PyTorch
tensors for the short calls, with the host compiler.  The module is made of
PyTorch's C++ classes, so it belongs to one version of PyTorch and of Python, which its
name holds: after a change of either it is built anew.  Without PyTorch
only the library is built.

Usage: ``python -m split_kv_merge_attn_b200._build`` (or ``build()``).  Both are
written next to this file so they travel with the source tree.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libsplitkv.so")

SOURCES = ["skv_kernels.cu", "skv_abi.cpp", "skv_noalloc.cu", "skv_cache.cu"]
HEADERS = ["skv_device.cuh", "skv_internal.h", "merge_state.cuh", "decode.cuh", "prefill.cuh",
           "smooth.cuh", "tcgen05.cuh", "quant.cuh", "rope.cuh", "kv8.cuh", "decode_kv8.cuh", "evict.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def command(out: str = LIB, extra=None):
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-shared",
           "-cudart", "static", "-t", "0", "-I", INCLUDE, "-I", CSRC]  # -t 0: the sources at the same time
    cmd += [os.path.join(CSRC, s) for s in SOURCES]
    cmd += ["-o", out]
    if extra:
        cmd += list(extra)
    return cmd


def torch_lib() -> str:
    """Path of the extension module for the PyTorch and Python that run."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(HERE, f"_skv_torch.torch-{torch.__version__}-abi{abi}{sysconfig.get_config_var('EXT_SUFFIX')}")


def torch_command(out: str):
    import torch
    from torch.utils import cpp_extension
    root = os.path.dirname(torch.__file__)
    include = cpp_extension.include_paths() + [os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
                                               sysconfig.get_paths()["include"]]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-Wall", "-I", INCLUDE]
    for p in include:
        cmd += ["-isystem", p]
    cmd += [os.path.join(CSRC, "skv_torch.cpp"), "-o", out, "-L", os.path.join(root, "lib")]
    return cmd + ["-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"]


def _stale(lib: str, deps) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in deps] + [os.path.join(INCLUDE, "splitkv.h"), __file__]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _run(cmd, name: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"building {name} failed")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr)


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    if force or _stale(LIB, SOURCES + HEADERS):
        _run(command(extra=extra), "libsplitkv.so", verbose)
    if importlib.util.find_spec("torch") is None:
        if verbose:
            print("PyTorch is not installed: only the C library is built")
    elif force or _stale(torch_lib(), ["skv_torch.cpp"]):
        _run(torch_command(torch_lib()), os.path.basename(torch_lib()), verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
