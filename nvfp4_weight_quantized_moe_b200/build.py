"""Build the sm_100a shared library ``libnvfp4moe.so`` in-tree with nvcc, and the
binding's small C++ part (``_quick_call``, against the installed PyTorch) with g++.
The library needs nvcc alone; without the C++ part the binding works through ctypes.

    python nvfp4_weight_quantized_moe_b200/build.py [--verbose-ptxas] [--force]

(run by path: importing the package first would load the library being rebuilt)

The library is a plain C ABI (include/nvfp4_moe.h) with the CUDA runtime
linked statically, so it loads with ctypes next to any PyTorch build.
"""

from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libnvfp4moe.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)

QUICK_SRC = os.path.join(CSRC, "quick_call.cpp")

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def needs_build() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps += glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def quick_call_path(torch_version: str) -> str:
    """Where the C++ part for this Python and that PyTorch lies: another version's, whose
    classes may be laid out differently, has another name and is not loaded."""
    return os.path.join(PKG_DIR, f"_quick_call.torch-{torch_version}" + sysconfig.get_config_var("EXT_SUFFIX"))


def build_quick_call(force: bool = False) -> str:
    """The binding's C++ part: the tensors' checks and the call without ctypes."""
    import torch
    path = quick_call_path(torch.__version__)
    deps = [QUICK_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps):
        return path
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(cuda, "include"),
           "-isystem", sysconfig.get_paths()["include"], "-I", INCLUDE, "-o", path + ".tmp", QUICK_SRC,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"g++ failed with exit code {res.returncode}")
    os.replace(path + ".tmp", path)
    return path


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """The library, and the binding's C++ part where its tools are there."""
    path = build_library(force, verbose_ptxas)
    try:
        build_quick_call(force)
    except (ImportError, OSError, RuntimeError) as e:  # no PyTorch, no g++, no headers
        sys.stderr.write(f"the binding's C++ part is not built ({e}): its calls go through ctypes\n")
    return path


def build_library(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not verbose_ptxas and not needs_build():
        return LIB_PATH
    cmd = [
        nvcc_path(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "--shared", "--threads", "0",
        "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC,
        "-DNVFP4_MOE_BUILD", "-o", LIB_PATH + ".tmp",
    ]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    cmd += sources()
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"nvcc failed with exit code {res.returncode}")
    if verbose_ptxas:
        sys.stdout.write(res.stderr)
    os.replace(LIB_PATH + ".tmp", LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--force", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose_ptxas=args.verbose_ptxas))
