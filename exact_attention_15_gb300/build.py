"""Builds the CUDA library in-tree: ``exact_attention_15_gb300/_lib/libattn_gb300.so``.

Every translation unit is compiled for sm_103a only (``-gencode
arch=compute_103a,code=sm_103a``), in parallel, and linked with the static CUDA
runtime, so the library needs nothing at load time but the C++ runtime (the
driver is reached lazily at the first call). Run ``python -m
exact_attention_15_gb300.build`` or call ``build()``.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libattn_gb300.so")
CALLS_LIB = os.path.join(LIBDIR, "_paged_call.so")

SOURCES = ["api.cu", "attn_fwd.cu", "attn_fwd_pair.cu", "attn_bwd.cu", "attn_bwd_pair.cu",
           "noalloc.cu", "paged_api.cu", "paged_append.cu", "paged_decode.cu", "paged_fwd.cu"]
CALLS = "paged_call.c"  # a CPython module: the paged cache's torch calls
HEADERS = ["ptx.cuh", "attn_common.cuh", "fwd_softmax.cuh", "host.h", "paged.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr"]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build")
    return cand


def _newest_dep_mtime():
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + [CALLS]]
    paths.append(os.path.join(ROOT, "include", "attn.h"))
    return max(os.path.getmtime(p) for p in paths if os.path.exists(p))


def _compile(src, extra):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_calls():
    """gcc for the CPython module (it includes no torch or CUDA header)."""
    tmp = CALLS_LIB + ".tmp"
    cmd = [shutil.which("gcc") or "cc", "-O2", "-Wall", "-shared", "-fPIC",
           "-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, CALLS), "-o", tmp, "-lm"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed for {CALLS}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS_LIB)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compiles and links the library if any source is newer than it. Returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    if (not force and os.path.exists(LIB) and os.path.exists(CALLS_LIB)
            and os.path.getmtime(LIB) >= _newest_dep_mtime()):
        return LIB
    extra = list(extra_flags)
    if verbose:
        extra += ["-Xptxas", "-v"]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_calls)
        results = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    calls.result()
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
