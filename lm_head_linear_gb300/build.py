"""In-tree build of the CUDA library ``_lib/libflce.so`` for sm_103a.

Plain ``nvcc``: a few translation units compiled side by side, one
``-gencode`` (compute_103a -> sm_103a), static CUDA runtime,
position-independent shared object.  Run as ``python -m lm_head_linear_gb300.build``.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG_DIR, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libflce.so")
SOURCES = [os.path.join(CSRC, f) for f in ("flce_api.cu", "flce_norm.cu", "flce_fp8.cu", "flce_losses.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in (
    "flce_host.cuh", "flce_kernels.cuh", "fp8_kernels.cuh", "loss_kernels.cuh", "norm_kernels.cuh", "ptx.cuh",
    "vec8.cuh")] + [
    os.path.join(INCLUDE, "flce.h")]

GENCODE = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def compile_command(src: str, obj: str, extra=()) -> list:
    return [nvcc_path(), GENCODE, "-O3", "-lineinfo", "-std=c++17",
            "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-c",
            "-I", INCLUDE, "-I", CSRC, *extra, "-o", obj, src]


def link_command(objs, out: str = LIB_PATH) -> list:
    return [nvcc_path(), GENCODE, "-shared", "-Xcompiler", "-fPIC", "-o", out, *objs]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in DEPENDS)


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr, flush=True)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile the library if any source is newer than it; returns its path."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB_PATH + ".tmp"
    objs = [os.path.join(LIB_DIR, os.path.basename(src) + ".o") for src in SOURCES]
    with ThreadPoolExecutor(len(SOURCES)) as pool:
        list(pool.map(lambda so: _run(compile_command(*so, extra), verbose), zip(SOURCES, objs)))
    _run(link_command(objs, tmp), verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
