"""Builds the in-tree C-ABI library ``libdsa_index.so`` for sm_100a.

Usage: ``python -m sparse_attention_token_index_b200.build [--verbose] [--debug-bounds]``.
Each ``csrc/*.cu`` is compiled with nvcc (``-gencode
arch=compute_100a,code=sm_100a``) in parallel and linked into one shared
library next to this file; the CUDA runtime is linked statically, so the
library loads without a GPU (only calls into it need one).  ``csrc/paged_ext.cpp``
becomes ``_paged_ext.so``, the Python extension that hands torch tensors to the
library's paged-cache calls; the library is built first and does without it.

``--debug-bounds`` builds ``libdsa_index_debug.so`` instead: the same
library compiled with ``-DDSA_DEBUG_BOUNDS=1``, whose kernels check the
indices that they compute for lists, caches, tables, partial results and
outputs against those buffers and record a failing check in the status word (``DSA_LIB`` selects it at load time).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdsa_index.so")
DEBUG_LIB = os.path.join(PKG, "libdsa_index_debug.so")
EXT = os.path.join(PKG, "_paged_ext.so")
EXT_SRC = os.path.join(CSRC, "paged_ext.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
    "-I" + INCLUDE, "-I" + CSRC,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
        os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build_ext(force: bool = False) -> str:
    """Compiles the Python extension against the installed torch: anew when a source has changed, and for another
    torch or Python than it was built for (a binary of one loads, or fails, in the other)."""
    import sysconfig

    import torch
    deps = [EXT_SRC, os.path.join(INCLUDE, "dsa_paged.h"), os.path.join(INCLUDE, "dsa_index.h"), __file__]
    key = f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"  # stands in the binary, as the module's __doc__
    if not force and os.path.exists(EXT) and all(os.path.getmtime(p) <= os.path.getmtime(EXT) for p in deps):
        with open(EXT, "rb") as f:
            if key.encode() in f.read():
                return EXT
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = EXT + ".tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DDSA_BUILT_FOR="{key}"',
           "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], f"-I{root}/include", f"-I{root}/include/torch/csrc/api/include",
           f"-I{cuda}/include", EXT_SRC, "-o", tmp, f"-L{root}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {EXT_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    return EXT


def build(verbose: bool = False, force: bool = False, extra_flags=None, debug_bounds: bool = False) -> str:
    lib = DEBUG_LIB if debug_bounds else LIB
    if force or not up_to_date(lib):
        _build_lib(lib, verbose, extra_flags, debug_bounds)
    try:
        build_ext(force and not debug_bounds)
    except (RuntimeError, OSError, ImportError) as e:  # no C++ compiler, no Python headers, no torch
        warnings.warn(f"{os.path.basename(lib)} is built, the Python extension is not: {e}", RuntimeWarning, stacklevel=2)
    return lib


def _build_lib(lib: str, verbose: bool, extra_flags, debug_bounds: bool) -> None:
    build_dir = BUILD + ("_debug" if debug_bounds else "")
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    flags = NVCC_FLAGS + (["-DDSA_DEBUG_BOUNDS=1"] if debug_bounds else []) + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, (r.stdout + r.stderr)

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, sources()))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = lib + ".tmp"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-cudart", "static",
           "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv,
                debug_bounds="--debug-bounds" in sys.argv))
