"""Build libfd.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc, and
_fdcall (Python's calls of a part of it, csrc/fdcall.c) with the C compiler."""
from __future__ import annotations

import glob
import os
import shlex
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfd.so")
# Named for the interpreter whose ABI it has.
CALLS = os.path.join(HERE, "_fdcall" + sysconfig.get_config_var("EXT_SUFFIX"))

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-Xptxas", "-v",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("CUDA_HOME") and os.path.join(os.environ["CUDA_HOME"], "bin", "nvcc"),
                 shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        os.path.join(ROOT, "include", "fd.h")]


def build_calls(force: bool = False) -> str:
    src, header = os.path.join(CSRC, "fdcall.c"), os.path.join(ROOT, "include", "fd.h")
    if (force or not os.path.exists(CALLS)
            or os.path.getmtime(CALLS) < max(os.path.getmtime(src), os.path.getmtime(header))):
        subprocess.check_call(shlex.split(os.environ.get("CC", "gcc")) + [
                              "-O2", "-Wall", "-Wextra", "-shared", "-fPIC",
                              "-I", os.path.join(ROOT, "include"),
                              "-I", sysconfig.get_paths()["include"], src, "-o", CALLS])
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu into split_kv_decode_attn_b200/libfd.so (skipped when
    the library is newer than every source), and csrc/fdcall.c beside it.  The
    library does not need the latter: where it cannot be built (no Python.h), its
    calls go through ctypes."""
    lib = build_library(force, verbose)
    try:
        build_calls(force)
    except (OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"{os.path.basename(CALLS)} could not be built ({e}); calls go through "
                      "ctypes, which takes a few microseconds more each")
    return lib


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(p) for p in deps())
        if os.path.getmtime(LIB) >= newest:
            return LIB
    cmd = [nvcc()] + NVCC_FLAGS + ["-I", os.path.join(ROOT, "include")] + sources() + ["-o", LIB]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed:\n{r.stdout}\n{r.stderr}")
    with open(os.path.join(HERE, "libfd.build.log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if verbose:
        print(r.stdout + r.stderr)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)
