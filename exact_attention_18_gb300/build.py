"""Compile the CUDA library in-tree for sm_103a.

The shared object lands in ``exact_attention_18_gb300/_lib/libfa_gb300.so``
(object files in ``_build/``); both are git-ignored.  Translation units are
compiled in parallel with one ``-gencode`` target, then linked with nvcc.
``_lib/_fa_binding.so``, the tensor binding of the serving calls, is host C++
against PyTorch's and Python's headers, linked to the library.  Where PyTorch is
not installed the library alone is built: it needs nvcc and nothing else.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libfa_gb300.so")
BINDING_SRC = os.path.join(CSRC, "fa_binding.cpp")
BINDING_PATH = os.path.join(LIB_DIR, "_fa_binding.so")
BINDING_FOR = os.path.join(BUILD_DIR, "fa_binding.for")  # what the binding was compiled against

SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_fwd4.cu", "fa_fwd4p.cu", "fa_bwd.cu", "fa_bwd_scores.cu", "fa_merge.cu", "fa_rope.cu", "fa_keep.cu",
           "fa_paged_d16.cu", "fa_paged_d32.cu", "fa_paged_d64.cu", "fa_paged_d128.cu",
           "fa_paged_scores_d16.cu", "fa_paged_scores_d32.cu", "fa_paged_scores_d64.cu", "fa_paged_scores_d128.cu",
           "fa_paged_merge.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE,
                 "-diag-suppress", "177"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != os.path.basename(BINDING_SRC)] + [os.path.join(INCLUDE, "fa.h")]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc()] + CFLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _torch_dir() -> str | None:
    """Where PyTorch is installed, found without importing it; None where it is not."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _binding_target(torch_dir: str) -> str:
    """The PyTorch and Python that a binding is compiled against."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"torch {version} in {torch_dir}, {sys.implementation.cache_tag} {sysconfig.get_paths()['include']}\n"


def _read(path: str) -> str | None:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _compile_binding(torch_dir: str, verbose: bool) -> str:
    """The tensor binding's object file."""
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD_DIR, "fa_binding.o")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE,
           "-I" + os.path.join(torch_dir, "include"),
           "-I" + os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + cuda_inc, "-c", BINDING_SRC, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on fa_binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str, torch_dir: str, verbose: bool) -> None:
    torch_lib = os.path.join(torch_dir, "lib")
    tmp = BINDING_PATH + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", obj, "-o", tmp, "-L" + LIB_DIR, "-lfa_gb300",
           "-Wl,-rpath,$ORIGIN", "-L" + torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the tensor binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_FOR, "w") as f:
        f.write(_binding_target(torch_dir))


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Build (if stale) the library, and where PyTorch is installed its tensor binding; returns the library's path."""
    torch_dir = _torch_dir()
    lib_stale = force or _stale(LIB_PATH, _deps())
    binding_stale = torch_dir is not None and (
        force or _stale(BINDING_PATH, [BINDING_SRC, os.path.join(INCLUDE, "fa.h")])
        or _read(BINDING_FOR) != _binding_target(torch_dir))
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, torch_dir, verbose) if binding_stale else None
        if lib_stale:
            _link_library(list(ex.map(lambda s: _compile(s, verbose), SOURCES)), verbose)
        # (the library is there by now, whatever becomes of the binding)
        if binding:
            _link_binding(binding.result(), torch_dir, verbose)
    if torch_dir is None and verbose:
        print("PyTorch is not installed: the library is built without its tensor binding", flush=True)
    return LIB_PATH


def _link_library(objs, verbose: bool) -> None:
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
