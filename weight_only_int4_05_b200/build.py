"""Build libawq_w4a16.so in-tree with nvcc for sm_100a (B200).

    python -m weight_only_int4_05_b200.build [--verbose]

The library links the CUDA runtime statically, so it needs only the NVIDIA driver at run time.  The CPython module _calls
(csrc/calls.c) is built beside it and linked against it; it saves about 1 us per call and needs a C compiler and Python.h,
so where it cannot be built the same calls go through ctypes.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_NAME = "libawq_w4a16.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
SOURCES = ["api.cu", "prep.cu", "pack.cu", "gemv.cu", "gemm.cu", "noalloc.cu", "selftest.cu", "search.cu", "gptq.cu",
           "fp8.cu", "w8a8.cu", "route.cu", "moe.cu"]
CALLS_SOURCE = "calls.c"
CALLS_PATH = os.path.join(PKG_DIR, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
HEADERS = ["common.cuh", "internal.h", "fp8.cuh", "w8a8.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


HEADER = os.path.join(ROOT, "include", "awq_w4a16.h")


def _newer(built: str, inputs) -> bool:
    return os.path.exists(built) and all(os.path.getmtime(f) <= os.path.getmtime(built) for f in inputs)


def _library_up_to_date() -> bool:
    return _newer(LIB_PATH, [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [HEADER])


def _calls_up_to_date() -> bool:
    return _newer(CALLS_PATH, [os.path.join(CSRC, CALLS_SOURCE), HEADER])


def up_to_date() -> bool:
    return _library_up_to_date() and _calls_up_to_date()


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not _library_up_to_date():
        _build_library(verbose)
    if force or not _calls_up_to_date():
        _build_calls()
    return LIB_PATH


def _build_library(verbose: bool) -> None:
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "--threads", "0",
           "-cudart", "static", f"-I{os.path.join(ROOT, 'include')}", "-o", tmp]
    if verbose:
        cmd.append("-Xptxas=-v")
    cmd += [os.path.join(CSRC, f) for f in SOURCES]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, LIB_PATH)


def _build_calls() -> None:
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    why = "no C compiler found"
    if cc:
        tmp = CALLS_PATH + f".{os.getpid()}.tmp"
        cmd = [cc, "-O2", "-Wall", "-shared", "-fPIC", f"-I{sysconfig.get_paths()['include']}",
               f"-I{os.path.join(ROOT, 'include')}", "-o", tmp, os.path.join(CSRC, CALLS_SOURCE), f"-L{PKG_DIR}",
               f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"]
        try:
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode == 0:
                os.replace(tmp, CALLS_PATH)
                return
            why = (res.stdout + res.stderr).strip()
        except OSError as e:
            why = str(e)
    if os.path.exists(CALLS_PATH):
        os.remove(CALLS_PATH)  # of an older source
    warnings.warn(f"the 8-bit operators' calls go through ctypes, _calls was not built: {why}", RuntimeWarning, stacklevel=3)


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
