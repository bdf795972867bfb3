"""Builds libep_gb300.so in-tree for sm_103a with nvcc, and beside it, where torch
is installed, the torch layer's compiled calls.

Each .cu file is compiled in its own nvcc process (in parallel), then the
objects are linked into one shared library with the CUDA runtime linked
statically.  ep_torch_calls (csrc/torch_calls.cpp) is a Python extension for
the installed torch, compiled by the host compiler and linked to that
library.  Usage: ``python combine_get_layout_gb300/build_lib.py [--force]``.
This file is standalone (it never imports the package, whose import needs the
built library).
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
OUT_DIR = os.path.join(PKG, "_lib")
BUILD_DIR = os.path.join(PKG, "_build_obj")
LIB = os.path.join(OUT_DIR, "libep_gb300.so")
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
HEADERS = [os.path.join(ROOT, "include", "ep.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden",
]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return sources() + HEADERS + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                                  if f.endswith((".cuh", ".h"))]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def calls_path():
    """ep_torch_calls for the installed torch, or None without one (with CUDA):
    one file a Python and torch, whose binary interfaces it follows."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None
    if not os.path.exists(os.path.join(torch_dir(), "lib", "libc10_cuda.so")):
        return None
    return os.path.join(OUT_DIR, "ep_torch_calls.%s.torch%s.so" % (
        sys.implementation.cache_tag, version.replace("+", ".")))


def calls_up_to_date(calls: str) -> bool:
    if not os.path.exists(calls):
        return False
    t = os.path.getmtime(calls)
    return all(os.path.getmtime(d) <= t for d in [CALLS_SRC, *HEADERS])


def compile_calls() -> str:
    """The object file of ep_torch_calls; linked after the library."""
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(nvcc()) or nvcc())))
    inc = [os.path.join(torch_dir(), "include"),
           os.path.join(torch_dir(), "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    obj = os.path.join(BUILD_DIR, "torch_calls.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", CALLS_SRC, "-o", obj]
    for d in inc:
        cmd += ["-isystem", d]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def link_calls(obj: str, calls: str) -> None:
    torch_lib = os.path.join(torch_dir(), "lib")
    tmp = calls + f".tmp{os.getpid()}"
    # torch's own libraries are loaded before the extension is, this one from
    # beside it
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L" + OUT_DIR, "-l:" + os.path.basename(LIB),
           "-Wl,-rpath,$ORIGIN", "-L" + torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {calls} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, calls)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    calls = calls_path()
    if not force and up_to_date():
        if calls is not None and not calls_up_to_date(calls):
            os.makedirs(BUILD_DIR, exist_ok=True)
            link_calls(compile_calls(), calls)
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        calls_obj = ex.submit(compile_calls) if calls is not None else None
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if calls_obj is not None:
        link_calls(calls_obj.result(), calls)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
