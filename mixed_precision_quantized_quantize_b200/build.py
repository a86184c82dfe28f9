"""Compile the CUDA library (sm_100a) in-tree: libquik_b200.so next to this file.

    python -m mixed_precision_quantized_quantize_b200.build [--force] [--verbose]

nvcc cross-compiles without a GPU.  The CUDA runtime is linked statically and
the driver API is reached through cudaGetDriverEntryPoint, so the library
loads on a machine without a GPU (no symbol needs libcuda at load time).
The library needs nvcc alone; the extension module _calls, which only the
attention's Python calls use, also needs torch and a C++ compiler, and is left
out where these are not there.
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libquik_b200.so")
# self-checking variant (-DQUIK_CHECKS): bounds checks that record and skip
LIB_CHECKED = os.path.join(HERE, "libquik_b200_checked.so")
# the attention calls from Python (a CPython extension over torch's C++ API)
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
CALLS = os.path.join(HERE, "_calls.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--shared", "-cudart", "static",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + [os.path.join(ROOT, "include", "quik.h"), __file__])


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def build_calls(force: bool = False) -> str:
    """The extension module _calls: host code only, for the torch that is installed."""
    deps = [CALLS_SRC, os.path.join(ROOT, "include", "quik.h"), __file__]
    if not force and os.path.exists(CALLS) and all(os.path.getmtime(d) <= os.path.getmtime(CALLS) for d in deps):
        return CALLS
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    tmp = CALLS + f".tmp{os.getpid()}"
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
        f'-DQUIK_TORCH_VERSION="{torch.__version__}"',
        "-I", os.path.join(base, "include"), "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
        "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
        # the C++ runtime before torch's libraries, which carry parts of one of their own
        CALLS_SRC, "-o", tmp, "-Wl,--no-as-needed", "-l:libstdc++.so.6", "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(tmp, CALLS)
    return CALLS


def build(force: bool = False, verbose: bool = False, checks: bool = False) -> str:
    lib = LIB_CHECKED if checks else LIB
    if force or not up_to_date(lib):
        _compile(lib, verbose, checks)
    if not checks:
        try:
            build_calls(force)
        except (ImportError, OSError, subprocess.CalledProcessError) as e:
            if os.path.exists(CALLS):  # of older sources: it must not meet the new library
                os.remove(CALLS)
            print(f"_calls is left out, the attention's Python calls will say so: {e}", file=sys.stderr)
    return lib


def _compile(lib: str, verbose: bool, checks: bool) -> None:
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, *(["-DQUIK_CHECKS"] if checks else []),
           "-I", os.path.join(ROOT, "include"), "-o", tmp, *sources()]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, lib)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--checks", action="store_true", help="build the self-checking variant")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, checks=a.checks))
