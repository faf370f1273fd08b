"""Compile libgqa_attn.so in-tree with nvcc for sm_103a, and the binding's extension.

The sources under ``csrc/`` are compiled in parallel, one object each, and
linked into ``_build/libgqa_attn.so`` next to this file. The CUDA runtime is
linked statically, so the library loads on a machine without a GPU driver
(the driver API is reached at run time through cudaGetDriverEntryPoint).

``csrc/binding.cpp`` becomes ``_build/_gqa_binding-torch<version>...so``, a Python extension
that only checks torch tensors and calls into the library (it links against torch, not against
it). It belongs to one version of torch and Python, and only the 4-bit cache's calls need it.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libgqa_attn.so")
EXT_SRC = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def ext_path() -> str:
    """The extension's file: one for each torch and Python, whose headers it was built from."""
    import torch
    return os.path.join(BUILD, f"_gqa_binding-torch{torch.__version__}"
                               f"{sysconfig.get_config_var('EXT_SUFFIX')}")


def ext_up_to_date() -> bool:
    if not os.path.exists(ext_path()):
        return False
    t = os.path.getmtime(ext_path())
    return all(os.path.getmtime(p) <= t for p in [EXT_SRC] + glob.glob(
        os.path.join(INCLUDE, "*.h")))


def build_ext(force: bool = False) -> str:
    """Build the binding's extension if it is older than its source; return its path."""
    out = ext_path()
    if not force and ext_up_to_date():
        return out
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    os.makedirs(BUILD, exist_ok=True)
    tmp = out + f".tmp{os.getpid()}"
    lib = os.path.join(root, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", EXT_SRC, "-o", tmp,
           "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-L", lib, f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}{r.stderr}")
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build the library and the extension if any source is newer; return the library's path."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        ext = ex.submit(build_ext, force)
        lib = build_lib(force, verbose, extra_flags)
        ext.result()
    return lib


def build_lib(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build the library if any source is newer than it; return its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = [nvcc()] + ARCH + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}{r.stderr}")
        return r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        logs = list(ex.map(compile_one, zip(srcs, objs)))
    if verbose:
        for s, lg in zip(srcs, logs):
            if lg.strip():
                print(f"--- {os.path.basename(s)}\n{lg}", file=sys.stderr)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else ()))
