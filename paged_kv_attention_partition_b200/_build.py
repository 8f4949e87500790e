"""Builds libpad.so in-tree with nvcc for sm_100a (cross-compiles without a GPU),
and the binding's argument marshalling for this torch (_pad_torch.*.so) with g++."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libpad.so")

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
SOURCES = ["pad_api.cpp", "pad_rows_api.cpp", "pad_shared_api.cpp", "pad_partition.cu", "pad_umma.cu", "pad_no_alloc.cu",
           "pad_rows.cu", "pad_shared.cu"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    files += glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return files


def is_stale(out: str = LIB) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(f) > t for f in _inputs())


def compile_command(out: str, extra=()):
    return [nvcc(), "-O3", "-std=c++17", *ARCH_FLAGS, "-lineinfo", "-Xcompiler", "-fPIC", "-shared",
            "-I", INCLUDE, "-I", CSRC, *extra, "-o", out] + [os.path.join(CSRC, s) for s in SOURCES]


def binding_path() -> str:
    """The binding's module for this Python and torch: a module of another torch may
    not load, or may load and read its tensors wrongly, so each has a name of its own."""
    import torch

    return os.path.join(PKG, f"_pad_torch.{sys.implementation.cache_tag}-torch{torch.__version__}.so")


def binding_command(out: str):
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], INCLUDE, os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{d}" for d in inc), os.path.join(CSRC, "pad_torch.cpp"), "-o", out, f"-L{os.path.join(root, 'lib')}",
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build_binding(force: bool = False) -> str:
    """Compile the binding's module if its source or pad.h is newer (or force)."""
    path = binding_path()
    inputs = [os.path.join(CSRC, "pad_torch.cpp"), os.path.join(INCLUDE, "pad.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in inputs):
        return path
    tmp = path + f".tmp{os.getpid()}"
    cmd = binding_command(tmp)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libpad.so, and then the binding's module where there is a torch to bind
    to, if any source is newer (or force)."""
    build_library(force, verbose)
    try:
        import torch  # noqa: F401
    except ImportError:
        return LIB
    build_binding(force)
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile libpad.so, which needs neither torch nor Python, if any source is newer (or force)."""
    if not force and not is_stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = compile_command(tmp, ["-Xptxas", "-v"] if verbose else [])
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
