"""Build libsta.so (the C-ABI STA library, nvcc for sm_100a) and _sta_torch.so (checks and
allocation of the prompt side's calls on PyTorch tensors; host code) in-tree."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG_DIR, "libsta.so")
# The same library with the device-side checks of every plan index compiled in
# (STA_DEBUG_BOUNDS; see csrc/sta_bounds.cuh).
DEBUG_LIB_PATH = os.path.join(PKG_DIR, "libsta_debug.so")

TORCH_PATH = os.path.join(PKG_DIR, "_sta_torch.so")
TORCH_SOURCE = os.path.join(CSRC, "sta_torch.cpp")
TORCH_STAMP = os.path.join(PKG_DIR, "_sta_torch.stamp")  # the torch_key that _sta_torch.so was built for

SOURCES = ["sta_api.cu", "sta_permute.cu", "sta_forward.cu", "sta_backward.cu", "sta_search.cu", "sta_pipe.cu", "sta_noalloc.cu",
           "sta_packed_lists.cu", "sta_packed.cu", "sta_packed_pair.cu",
           "sta_packed_backward.cu", "sta_cache.cu", "sta_cache_attention.cu"]
HEADERS = ["sta_internal.h", "sta_ptx.cuh", "sta_raster.cuh", "sta_wait.cuh", "sta_bounds.cuh",
           "sta_ops.h", "sta_ops.cuh", "sta_packed.cuh", "sta_packed_fwd.cuh"]

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared",
]


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(INCLUDE, "sta.h"))
    return files


def up_to_date(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _compile(path: str, extra, verbose: bool):
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = path + f".tmp{os.getpid()}"
    cmd = [nvcc, "--threads", "0", *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC,
           *[os.path.join(CSRC, f) for f in SOURCES], "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, path)


def torch_key() -> str:
    """The PyTorch and Python whose ABI _sta_torch.so has to be built for."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def _torch_command(out: str):
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f'-DSTA_TORCH_KEY="{torch_key()}"', *[a for i in inc for a in ("-isystem", i)], TORCH_SOURCE, "-o", out, "-L", os.path.join(torch_dir, "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]


def _torch_up_to_date() -> bool:
    if not os.path.exists(TORCH_PATH) or not os.path.exists(TORCH_STAMP):
        return False
    with open(TORCH_STAMP) as f:
        if f.read() != torch_key():
            return False
    return all(os.path.getmtime(f) <= os.path.getmtime(TORCH_PATH) for f in (TORCH_SOURCE, os.path.join(INCLUDE, "sta.h")))


def _build_torch(verbose: bool):
    tmp = TORCH_PATH + f".tmp{os.getpid()}"
    cmd = _torch_command(tmp)
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, TORCH_PATH)
    with open(TORCH_STAMP, "w") as f:
        f.write(torch_key())


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Build libsta.so and _sta_torch.so (and, with debug=True, also libsta_debug.so)."""
    if force or not _torch_up_to_date():
        _build_torch(verbose)
    if force or not up_to_date(LIB_PATH):
        _compile(LIB_PATH, [], verbose)
    if debug and (force or not up_to_date(DEBUG_LIB_PATH)):
        _compile(DEBUG_LIB_PATH, ["-DSTA_DEBUG_BOUNDS"], verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
