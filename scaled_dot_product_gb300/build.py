"""Builds libsdpa.so in-tree with nvcc for sm_103a (no cmake).

Each translation unit under csrc/ is compiled in parallel to an object in _build/,
then linked into scaled_dot_product_gb300/libsdpa.so; csrc/binding.cpp, the native part of the
Python binding, becomes scaled_dot_product_gb300/_binding.so.  Up-to-date objects are reused.
The library needs neither torch nor its headers: it is built where the binding cannot be.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsdpa.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libsdpa")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


# The bounds-checking debug build: every guarded index is range-checked in the kernels; a
# failed check records its site (sdpa_query_status: SDPA_ERR_BOUNDS) and skips the access.
LIB_BOUNDS = os.path.join(PKG, "libsdpa_bounds.so")


# The marshalling module of sdpa.py (Python's and torch's C++ headers; no CUDA).
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")


def build_binding(verbose: bool = False) -> str:
    """Builds the binding; raises if it cannot, and leaves no older one in its place."""
    try:
        return _build_binding(verbose)
    except Exception:
        if os.path.exists(BINDING):
            os.remove(BINDING)
        raise


def _build_binding(verbose: bool) -> str:
    import torch
    root = os.path.dirname(torch.__file__)
    # built against one interpreter and one torch: a stamp names them
    stamp = os.path.join(BUILD, "binding.stamp")
    what = f"{sys.version}\n{torch.__version__}\n"
    old = open(stamp).read() if os.path.exists(stamp) else ""
    if old == what and not _stale(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "sdpa.h"), __file__]):
        return BINDING
    os.makedirs(BUILD, exist_ok=True)
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", BINDING_SRC, "-o", tmp,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"), "-L", os.path.join(root, "lib"),
           "-lc10", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(what)
    return BINDING


def build(verbose: bool = False, extra_flags=None, bounds_check: bool = False) -> str:
    """Builds the library and returns its path; the binding too, where it can be (what kept it from
    that is printed, and the norm and paged calls of sdpa.py raise without it)."""
    nvcc = _nvcc()
    build_dir = BUILD + ("_bounds" if bounds_check else "")
    lib_path = LIB_BOUNDS if bounds_check else LIB
    os.makedirs(build_dir, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    flags = FLAGS + list(extra_flags or []) + (["-DSDPA_BOUNDS_CHECK"] if bounds_check else [])

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        if _stale(obj, [src] + headers + [__file__]):
            cmd = [nvcc] + ARCH + flags + ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
            if verbose and r.stderr:
                print(r.stderr, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(sources) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(build_binding, verbose)
        objs = list(ex.map(compile_one, sources))
    if _stale(lib_path, objs):
        tmp = lib_path + f".tmp{os.getpid()}"
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, lib_path)
    if binding.exception() is not None:
        print(f"{lib_path} is built, {BINDING} is not: {binding.exception()}", file=sys.stderr)
    return lib_path


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, bounds_check="--bounds-check" in sys.argv))
