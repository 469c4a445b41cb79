"""Build libsvdq.so (sm_100a) in-tree with nvcc.

    python -m bit_w4a4_quantized_group_b200.build [--verbose] [--debug]

Each source under ``csrc/`` is compiled to an object in ``_build/`` (in
parallel), then linked into ``_lib/libsvdq.so`` with the CUDA runtime linked
statically.  ``csrc/svdq_call.c`` becomes ``_lib/svdq_call.so``, the binding's CPython extension.  No GPU is needed to build.

``--debug`` builds ``_lib/libsvdq_debug.so`` instead (objects in ``_build_debug/``):
the same kernels compiled with -DSVDQ_DEBUG, in which every plain global or
shared-memory access of the kernels checks its index first; an access that
would fall outside its buffer is skipped and recorded in the device error word
(sites 201 and 202 of svdq_get_last_device_error).
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
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libsvdq.so")
CALLS = os.path.join(LIBDIR, "svdq_call.so")      # CPython extension of the binding, see csrc/svdq_call.c
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(LIBDIR, "libsvdq_debug.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    srcs = []
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cpp")):
            srcs.append(os.path.join(CSRC, f))
    return srcs


def _deps_mtime():
    m = 0.0
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            m = max(m, os.path.getmtime(os.path.join(d, f)))
    return m


def _compile(src: str, verbose: bool, debug: bool = False) -> str:
    obj = os.path.join(BUILD_DEBUG if debug else BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *COMMON, *(["-DSVDQ_DEBUG"] if debug else []), "-c", src, "-o", obj]
    if src.endswith(".cu"):
        cmd += ["-lineinfo"]
        if verbose:
            cmd += ["-Xptxas", "-v"]
    else:
        cmd += ["-x", "c++"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _python_include() -> str:
    """Directory of Python.h, or "" where Python's headers are not installed."""
    inc = sysconfig.get_paths()["include"]
    return inc if os.path.exists(os.path.join(inc, "Python.h")) else ""


def _build_calls(force: bool = False) -> None:
    """The binding's extension, unless it is up to date.  It is optional: without Python's headers or a C
    compiler that takes it the binding goes through ctypes alone, and an extension built from an older
    source, whose calls need not match the library any more, is taken away."""
    src = os.path.join(CSRC, "svdq_call.c")
    if not force and os.path.exists(CALLS) and os.path.getmtime(CALLS) >= max(
            os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "svdq.h"))):
        return
    inc, why = _python_include(), "Python.h not found"
    if inc:
        tmp = CALLS + ".tmp"
        try:
            r = subprocess.run(["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I", inc, "-I", INCLUDE, src, "-o", tmp],
                               capture_output=True, text=True)
            if r.returncode == 0:
                os.replace(tmp, CALLS)
                return
            why = r.stdout + r.stderr
        except OSError as e:
            why = str(e)
    sys.stderr.write(f"svdq_call.so not built, the binding uses ctypes alone: {why}\n")
    if os.path.exists(CALLS):
        os.remove(CALLS)


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile every CUDA / C++ source of the library for sm_100a; return the .so path
    (the bounds-checking debug library when debug is true)."""
    lib = LIB_DEBUG if debug else LIB
    os.makedirs(LIBDIR, exist_ok=True)
    if not debug:
        _build_calls(force)
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= _deps_mtime():
        return lib
    os.makedirs(BUILD_DEBUG if debug else BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, debug), srcs))
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv, debug="--debug" in sys.argv))
