"""Builds libfa.so (the C-ABI attention library) in-tree with nvcc for sm_100a, and the quick
binding of its serving calls (_fa_binding.so) with g++ against torch's headers.

Usage:  python -m exact_io_aware_60_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfa.so")
BINDING = os.path.join(PKG, "_fa_binding.so")
BINDING_STAMP = os.path.join(PKG, "_fa_binding.stamp")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-Xptxas", "-v",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, "fa.h")])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def binding_command(out: str):
    """(command, stamp): the stamp names all that the binding is compiled against, the sources
    aside; it reads tensors through torch's own classes, whose layout is a version's."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DFA_TORCH_VERSION="{torch.__version__}"', f"-I{INCLUDE}",
           *(f"-I{p}" for p in ext.include_paths(device_type="cuda")),
           f"-I{sysconfig.get_paths()['include']}", BINDING_SRC, "-o", out,
           *(f"-L{p}" for p in ext.library_paths(device_type="cuda")),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    flags = [x for x in cmd if x.startswith(("-O", "-D", "-s", "-f", "-l"))]
    return cmd, " ".join([torch.__version__, sysconfig.get_config_var("SOABI") or "", *flags]) + "\n"


def binding_up_to_date(stamp: str) -> bool:
    try:
        with open(BINDING_STAMP) as f:
            if f.read() != stamp:
                return False
        t = os.path.getmtime(BINDING)
    except OSError:
        return False
    return all(os.path.getmtime(s) <= t for s in (BINDING_SRC, os.path.join(INCLUDE, "fa.h")))


def build_binding(force: bool = False, verbose: bool = False) -> str:
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd, stamp = binding_command(tmp)
    if not force and binding_up_to_date(stamp):
        return BINDING
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError("g++ failed building _fa_binding.so")
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(stamp)
    return BINDING


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC,
           os.path.join(CSRC, "fa_api.cu"), "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed building libfa.so")
    # ptxas resource report (registers, spills, shared memory) kept beside the library
    with open(os.path.join(PKG, "libfa.ptxas.txt"), "w") as f:
        f.write(res.stderr)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds the library, which needs nvcc alone, and then the quick binding.  Without the binding
    (no g++, torch or Python headers) the same calls go by ctypes, so that its failure is said and
    nothing more."""
    build_library(force, verbose)
    try:
        build_binding(force, verbose)
    except Exception as e:  # noqa: BLE001 -- whatever it was, the library stands
        sys.stderr.write(f"_fa_binding.so not built ({type(e).__name__}: {e}); the serving calls "
                         "go by ctypes, some 5 us of host time each slower\n")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
