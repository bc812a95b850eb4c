"""Builds the CUDA library libmha.so in-tree with nvcc for sm_103a, and beside it
the inner part of the Python binding (binding.cpp) with the host compiler.

Each translation unit is compiled in parallel, then linked into one shared
library against the shared CUDA runtime (the one PyTorch already loaded).
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmha.so")


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return "unknown"


# of this PyTorch and interpreter alone: others do not find it, and do without
BINDING = os.path.join(BUILD, "_mha_binding.torch-%s%s" % (
    _torch_version(), sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

SOURCES = ["mha_api.cu", "attn_f32_simt.cu", "attn_short_tc.cu", "attn_long_tc.cu", "attn_decode_tc.cu",
           "attn_bwd_simt.cu", "attn_bwd_tc.cu", "linear_tc.cu", "paged_api.cu", "qk_rope.cu",
           "paged_simt.cu", "paged_few_tc.cu", "paged_many_tc.cu", "pages_api.cu", "pages_reserve.cu",
           "pages_move.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _fresh(path: str) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()


def build_binding(verbose: bool = False) -> bool:
    """Compile binding.cpp against PyTorch's headers; False (and no file) where that is
    not possible: the binding then makes its checks and calls in Python."""
    spec = importlib.util.find_spec("torch")
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    with contextlib.suppress(FileNotFoundError):
        os.remove(BINDING)
    if spec is None or not spec.submodule_search_locations or cxx is None:
        return False
    torch = spec.submodule_search_locations[0]
    tmp = BINDING + ".tmp.%d" % os.getpid()
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-D_GLIBCXX_USE_CXX11_ABI=1",
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch, "include"),
           "-I", INCLUDE, os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        print("binding.cpp not built, calls are made through ctypes:\n" + res.stderr[-2000:],
              file=sys.stderr)
        return False
    if verbose and res.stderr:
        print(res.stderr)
    os.replace(tmp, BINDING)
    return True


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (if stale) and return the path of libmha.so."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # beside the library's own files
        binding = None if _fresh(BINDING) and not force else ex.submit(build_binding, verbose)
        if force or not _fresh(LIB):
            _build_library(verbose, extra_flags)
        if binding is not None:
            binding.result()
    return LIB


def _build_library(verbose: bool, extra_flags) -> None:
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr))
        if verbose and res.stderr:
            print(res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr))
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
