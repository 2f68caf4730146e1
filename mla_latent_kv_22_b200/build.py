"""Builds libmla.so in-tree with nvcc for sm_100a (B200), and the binding's quick path (an
extension module named after the torch and Python it is for) with g++ against torch's headers.

    python mla_latent_kv_22_b200/build.py [--force] [--verbose] [--ptxas]

(Run it as a file, not with ``-m``: importing the package loads the library.)
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmla.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-O3,-Wall",
    "-shared",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _newer(target: str, deps: list[str]) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def binding_path() -> str:
    """The quick path's extension for the running Python and torch.  It reads torch's C++
    objects, so one built for another version must never be loaded: each has a file of its own."""
    import torch

    tag = f"torch-{torch.__version__}-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(PKG, f"_binding.{tag}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _binding_up_to_date() -> bool:
    return _newer(binding_path(), [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and _binding_up_to_date()


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _run(cmd: list[str], target: str, verbose: bool) -> None:
    """Runs a compiler whose output goes to target + ".tmp", then moves it into place."""
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"{cmd[0]} failed building {os.path.basename(target)}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr)
    os.replace(target + ".tmp", target)


def _build_binding(verbose: bool) -> None:
    import torch

    T, target = os.path.dirname(torch.__file__), binding_path()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", INCLUDE, "-isystem", os.path.join(T, "include"), "-isystem", os.path.join(T, "include/torch/csrc/api/include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-o", target + ".tmp", BINDING_SRC, "-L", PKG, "-l:libmla.so",
          "-L", os.path.join(T, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
          "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + os.path.join(T, "lib")], target, verbose)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if force or not _newer(LIB, _deps()):
        _run([nvcc(), *NVCC_FLAGS, *(extra or []), "-I", INCLUDE, "-I", CSRC, "-o", LIB + ".tmp", *sources()], LIB, verbose)
    if force or not _binding_up_to_date():
        _build_binding(verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
          extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None)
