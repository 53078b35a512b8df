"""Build libspecverify.so in-tree with nvcc for sm_103a (GB300).

Each translation unit under csrc/ (CUDA .cu, host-only .cpp) compiles in its
own nvcc process, in parallel; the objects link into one shared library with the CUDA runtime
linked statically. csrc/torch_calls.cpp becomes the extension module _calls (g++,
against the installed torch's headers). Rebuilds only when a source or header is
newer than the built files, one of them is missing, or another torch is installed.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libspecverify.so")
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_FOR = os.path.join(BUILD, "calls_for")  # what _calls.so was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _sources():
    return sorted(set(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp"))) - {CALLS_SRC})


def _deps():
    return _sources() + [CALLS_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def _torch_here() -> str:
    """The torch and the interpreter that _calls.so has to fit."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def calls_fit() -> bool:
    """Whether _calls.so is there and was built against the torch that is installed."""
    if not os.path.exists(CALLS) or not os.path.exists(CALLS_FOR):
        return False
    with open(CALLS_FOR) as f:
        return f.read() == _torch_here()


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not calls_fit():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return all(os.path.getmtime(p) <= t for p in _deps())


def build_calls() -> None:
    """The extension module _calls, against the torch that is installed."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as X
    gxx = os.environ.get("CXX") or shutil.which("g++")
    if not gxx:
        raise RuntimeError("g++ not found: the Python bindings cannot be built")
    os.makedirs(BUILD, exist_ok=True)
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = [gxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], *("-I" + p for p in X.include_paths()), CALLS_SRC, "-o", tmp,
           *("-L" + p for p in X.library_paths()), "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(CALLS_SRC)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS_FOR, "w") as f:
        f.write(_torch_here())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        calls = ex.submit(build_calls)
        objs = list(ex.map(compile_one, srcs))
        calls.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
