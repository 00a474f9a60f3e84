"""Build libfa_gb300.so in-tree from csrc/*.cu with nvcc for sm_103a.

One translation unit per kernel family, compiled in parallel, then linked
into a shared library next to this file; and, where Python's headers are, the CPython
module _paged_calls, with the host's C compiler.  No torch C++ ABI is involved, so the same sources build on x86 and
Arm hosts.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libfa_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = ["fa_api.cu", "fa_prefill_sm103.cu", "fa_decode_sm103.cu", "fa_backward_sm103.cu",
           "fa_paged_api.cu", "fa_paged_sm103.cu", "fa_paged_tiles_sm103.cu",
           "fa_paged_cluster_sm103.cu", "fa_cache_sm103.cu", "fa_tree_sm103.cu", "fa_weigh_sm103.cu",
           "fa_weigh_tiles_sm103.cu", "fa_evict_sm103.cu"]
# The CPython module in front of the paged-cache calls (host code only).
CALLS_SOURCE = "paged_calls.c"
CALLS_PATH = os.path.join(HERE, "_paged_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
          "-Xcompiler", "-Wall"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand) and not shutil.which(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa_gb300.so")
    return cand


def _inputs_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(HERE, "..", "include", "fa.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _build_calls(verbose: bool) -> None:
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        # (the library needs none of it, and binding.py makes the same calls in Python)
        if os.path.exists(CALLS_PATH):
            os.remove(CALLS_PATH)  # of older sources
        sys.stderr.write(f"no Python.h in {include}: paged-cache calls stay in Python, some 3 us slower each\n")
        return
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        raise RuntimeError("a C compiler is required to build _paged_calls")
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([cc, "-O2", "-std=c11", "-Wall", "-shared", "-fPIC", "-I", include,
                        os.path.join(CSRC, CALLS_SOURCE), "-o", tmp, "-lm"], capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{cc} failed on {CALLS_SOURCE}")
    os.replace(tmp, CALLS_PATH)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if stale) and return the path of libfa_gb300.so."""
    newest = _inputs_mtime()
    _build_library(force, verbose, ptxas_info, newest)
    if force or not os.path.exists(CALLS_PATH) or os.path.getmtime(CALLS_PATH) < newest:
        _build_calls(verbose)
    return LIB_PATH


def _build_library(force: bool, verbose: bool, ptxas_info: bool, newest: float) -> None:
    if not force and os.path.exists(LIB_PATH) and os.path.getmtime(LIB_PATH) >= newest:
        return
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH_FLAGS, *COMMON, *extra, "-I", os.path.join(HERE, "..", "include"),
               "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    for src, _, r in results:
        if verbose or ptxas_info or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}")
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH_FLAGS, "-shared", "-o", tmp, *[o for _, o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("linking libfa_gb300.so failed")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB_PATH)
