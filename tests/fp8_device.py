"""Builds fp8_device.cu with the library's headers and flags, and loads it."""
import ctypes
import functools
import os
import subprocess
import tempfile

from weight_only_int4_05_b200 import build as libbuild


@functools.lru_cache(maxsize=None)
def load():
    here = os.path.dirname(os.path.abspath(__file__))
    out = os.path.join(tempfile.mkdtemp(prefix="fp8_device_"), "fp8_device.so")
    cmd = [libbuild.nvcc(), *libbuild.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-cudart", "static",
           f"-I{libbuild.CSRC}", f"-I{os.path.join(libbuild.ROOT, 'include')}", "-o", out, os.path.join(here, "fp8_device.cu")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    lib = ctypes.CDLL(out)
    lib.silu_of.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    lib.signal_then_run.argtypes = [ctypes.c_ulonglong, ctypes.c_void_p]
    return lib
