"""Build libkvx.so (the C-ABI library) in-tree for sm_103a with nvcc.

One object per translation unit, compiled in parallel: the transfer kernels (kvx.cu), page
upkeep (kvx_pages.cu), attention (kvx_attend.cu, over a 4-bit cache kvx_attend_four.cu), rotated
append (kvx_rotate.cu) and beam selection (kvx_beams.cu) by nvcc, the host logic (kvx_host.cpp,
kvx_cache_host.cpp) and the SM partitioning (kvx_partition.cpp) by the host C++ compiler.
The CUDA runtime is
linked statically so the library loads on machines without a GPU (its host logic and
exported symbols stay usable there).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libkvx.so")
BUILD_DIR = os.path.join(ROOT, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CUDA_UNITS = ("kvx.cu", "kvx_pages.cu", "kvx_attend.cu", "kvx_attend_four.cu",
              "kvx_rotate.cu", "kvx_beams.cu")
HOST_UNITS = ("kvx_host.cpp", "kvx_cache_host.cpp", "kvx_partition.cpp")
SOURCES = [os.path.join(CSRC, f) for f in CUDA_UNITS + HOST_UNITS + (
    "kvx_kernels.cuh", "kvx_internal.h", "kvx_rules.h", "kvx_ctx.h", "kvx_cache.h",
    "kvx_attend.cuh", "kvx_attend_rows.cuh", "kvx_attend_tiles.cuh", "kvx_attend_four.cuh",
    "kvx_attend_plan.h")]
HEADER = os.path.join(ROOT, "include", "kvx.h")


def cuda_home() -> str:
    for cand in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return cand
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    raise RuntimeError("nvcc not found: set CUDA_HOME")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in SOURCES + [HEADER])


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"build failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libkvx.so if a source is newer than it (or force); return its path."""
    if not force and not _stale():
        return LIB
    home = cuda_home()
    nvcc = os.path.join(home, "bin", "nvcc")
    inc = os.path.join(home, "include")
    os.makedirs(BUILD_DIR, exist_ok=True)
    tag = f"{os.getpid()}"
    cxx = shutil.which("g++") or shutil.which("c++")
    objs, cmds = [], []
    for src in CUDA_UNITS:
        obj = os.path.join(BUILD_DIR, f"{src[:-3]}.{tag}.o")
        objs.append(obj)
        cmds.append([nvcc, "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xptxas", "-v", "-Xcompiler",
                     "-fPIC", "-c", os.path.join(CSRC, src), "-o", obj])
    for src in HOST_UNITS:
        obj = os.path.join(BUILD_DIR, f"{src[:-4]}.{tag}.o")
        objs.append(obj)
        cmds.append([cxx, "-O2", "-std=c++17", "-fPIC", f"-I{inc}", "-c",
                     os.path.join(CSRC, src), "-o", obj])
    with ThreadPoolExecutor(len(cmds)) as ex:
        logs = list(ex.map(_run, cmds))
    tmp = LIB + f".tmp{tag}"
    _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)
    if verbose:
        sys.stdout.write("".join(logs[:len(CUDA_UNITS)]))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
