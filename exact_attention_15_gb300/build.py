"""Builds the CUDA library in-tree: ``exact_attention_15_gb300/_lib/libattn_gb300.so``.

Every translation unit is compiled for sm_103a only (``-gencode
arch=compute_103a,code=sm_103a``), in parallel, and linked with the static CUDA
runtime, so the library needs nothing at load time but the C++ runtime (the
driver is reached lazily at the first call). Run ``python -m
exact_attention_15_gb300.build`` or call ``build()``.

Beside it a small CPython module is built that makes the paged cache's common calls
(``csrc/paged_call.c``). It needs Python's headers; where they are missing the build says
so and goes on, and ``paged.py`` makes every call by itself.
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
# (named for the Python it was built for: another one builds its own)
CALLS_LIB = os.path.join(LIBDIR, "_paged_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

SOURCES = ["api.cu", "attn_fwd.cu", "attn_fwd_pair.cu", "attn_bwd.cu", "attn_bwd_pair.cu",
           "noalloc.cu", "paged_api.cu", "paged_append.cu", "paged_append_pages.cu", "paged_decode.cu", "paged_fwd.cu",
           "paged_select.cu"]
CALLS = "paged_call.c"  # a CPython module: the paged cache's torch calls
HEADERS = ["ptx.cuh", "attn_common.cuh", "fwd_softmax.cuh", "host.h", "paged.cuh", "append.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr"]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build")
    return cand


def _newest_dep_mtime(files):
    paths = [os.path.join(CSRC, f) for f in files]
    paths.append(os.path.join(ROOT, "include", "attn.h"))
    return max(os.path.getmtime(p) for p in paths if os.path.exists(p))


def _fresh(target, files):
    return os.path.exists(target) and os.path.getmtime(target) >= _newest_dep_mtime(files)


def _compile(src, extra):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _build_calls():
    """The CPython module, by the host's C compiler (it includes no torch or CUDA header).
    Where it cannot be built none is left, so that none of an older source is loaded."""
    tmp = CALLS_LIB + ".tmp"
    cmd = [shutil.which("gcc") or "cc", "-O2", "-Wall", "-shared", "-fPIC",
           "-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, CALLS), "-o", tmp, "-lm"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        said = None if r.returncode == 0 else r.stderr
    except OSError as e:
        said = str(e)
    if said is None:
        os.replace(tmp, CALLS_LIB)
        return
    if os.path.exists(CALLS_LIB):
        os.remove(CALLS_LIB)
    sys.stderr.write(f"{CALLS} was not built, the paged cache's calls are made from Python:\n{said}\n")


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compiles and links the library, and the CPython module, where a source is newer.
    Returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    if force or not _fresh(CALLS_LIB, [CALLS]):
        _build_calls()
    if not force and _fresh(LIB, SOURCES + HEADERS):
        return LIB
    extra = list(extra_flags)
    if verbose:
        extra += ["-Xptxas", "-v"]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(lambda s: _compile(s, extra), SOURCES))
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
