"""In-tree build of the CUDA library ``_lib/libflce.so`` for sm_103a, and of the
Python module ``_lib/flce_ops.so`` that calls its operators.

Plain ``nvcc``: a few translation units compiled side by side, one
``-gencode`` (compute_103a -> sm_103a), static CUDA runtime,
position-independent shared object.  The module is host C++ against torch's
headers, linked to the library; where it does not build, the library still does.
Run as ``python -m lm_head_linear_gb300.build``.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
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

OPS_SOURCE = os.path.join(CSRC, "ops_binding.cpp")
OPS_PATH = os.path.join(LIB_DIR, "flce_ops.so")

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


def ops_commands(obj: str, out: str) -> list:
    """Compile and link commands of the Python module (host compiler, torch's headers and libraries)."""
    import torch
    from torch.utils import cpp_extension
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    abi = int(torch.compiled_with_cxx11_abi())
    dirs = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [[cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-c",
             *(f"-isystem{d}" for d in dirs), "-o", obj, OPS_SOURCE],
            [cxx, "-shared", "-o", out, obj, f"-L{libs}", f"-L{LIB_DIR}", "-lflce", "-lc10", "-lc10_cuda", "-ltorch_cpu",
             "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]]


def running() -> str:
    """What the compiled Python module depends on besides its sources: torch's C++ interface has no stable ABI."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def ops_built_for() -> str:
    """running() as it was when the module was built ("" if that is not known)."""
    try:
        with open(OPS_PATH + ".for") as fh:
            return fh.read()
    except OSError:
        return ""


def up_to_date() -> bool:
    if not (os.path.exists(LIB_PATH) and os.path.exists(OPS_PATH) and ops_built_for() == running()):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in DEPENDS) and all(
        os.path.getmtime(f) <= os.path.getmtime(OPS_PATH) for f in (OPS_SOURCE, os.path.join(INCLUDE, "flce.h")))


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr, flush=True)


def _compile_ops(obj: str, out: str, verbose: bool) -> list:
    """Compiles the Python module; returns its link command."""
    compile_cmd, link_cmd = ops_commands(obj, out)
    _run(compile_cmd, verbose)
    return link_cmd


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile the library if any source is newer than it; returns its path.

    The library needs nvcc alone.  Where the Python module cannot be built (torch's headers or libraries, or
    Python's, are missing) a warning says why, and :func:`.ops.load_operators` raises."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp, ops_tmp = LIB_PATH + ".tmp", OPS_PATH + ".tmp"
    objs = [os.path.join(LIB_DIR, os.path.basename(src) + ".o") for src in SOURCES]
    with ThreadPoolExecutor(len(SOURCES) + 1) as pool:
        ops = pool.submit(_compile_ops, os.path.join(LIB_DIR, "ops_binding.o"), ops_tmp, verbose)
        list(pool.map(lambda job: _run(compile_command(*job, extra), verbose), zip(SOURCES, objs)))
    _run(link_command(objs, tmp), verbose)
    os.replace(tmp, LIB_PATH)
    try:
        _run(ops.result(), verbose)
        os.replace(ops_tmp, OPS_PATH)
        with open(OPS_PATH + ".for", "w") as fh:
            fh.write(running())
    except Exception as e:  # whatever torch's build helpers raise where something is missing
        if os.path.exists(OPS_PATH):
            os.remove(OPS_PATH)  # an older one, of another interface
        warnings.warn(f"{LIB_PATH} is built; {OPS_PATH} could not be: {e}")
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
