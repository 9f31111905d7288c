"""ctypes loader for libawq_w4a16.so (the C ABI of include/awq_w4a16.h).

Loading fails loudly when the shared library has not been built: there is no fallback path.  (The CPython module of the 8-bit
operators' calls has one, by ctypes into the same library.)
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading

from . import build as _build

EXPORTS = (
    "awq_status_string", "awq_version", "awq_packed_sizes", "awq_act_scale", "awq_apply_inv_scale",
    "awq_pack", "w4a16_gemv", "w4a16_gemm", "w4a16_linear", "w4a16_gemv_max_m", "w4a16_workspace_bytes",
    "awq_last_device_status", "w4a16_gemv_noalloc", "awq_selftest_wait_timeout",
    "w4a16_linear_pf", "w4a16_gemv_s", "awq_pack_gate_up", "w4a16_gate_up_silu", "awq_search_scale",
    "awq_search_workspace_bytes", "gptq_quantize", "gptq_workspace_bytes", "awq_pack_bits", "awq_packed3_sizes",
    "awq_pack3", "w3a16_gemv", "fp8_scale_bytes", "fp8_quantize", "w8a8_gemm", "w8a8_linear", "w8a8_workspace_bytes",
    "moe_route", "w8a8_moe", "w8a8_moe_workspace_bytes",
)

STATUS_NAMES = {0: "AWQ_OK", 1: "AWQ_ERR_INVALID_ARG", 2: "AWQ_ERR_UNSUPPORTED", 3: "AWQ_ERR_MISALIGNED",
                4: "AWQ_ERR_CUDA", 5: "AWQ_ERR_DEVICE_TIMEOUT", 6: "AWQ_ERR_WORKSPACE", 7: "AWQ_ERR_NUMERIC"}
MODE_GEMV, MODE_GEMM, MODE_LINEAR = 1, 2, 3

_lock = threading.Lock()
_lib = None


class AwqError(RuntimeError):
    def __init__(self, where: str, status: int):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


def lib_path() -> str:
    return _build.LIB_PATH


def load() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m weight_only_int4_05_b200.build`")
        lib = ctypes.CDLL(path)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.awq_status_string.restype = ctypes.c_char_p
        lib.awq_status_string.argtypes = [I]
        lib.awq_version.restype = I
        lib.awq_version.argtypes = []
        lib.awq_packed_sizes.restype = I
        lib.awq_packed_sizes.argtypes = [I, I, I, ctypes.POINTER(Z), ctypes.POINTER(Z), ctypes.POINTER(Z)]
        lib.awq_act_scale.restype = I
        lib.awq_act_scale.argtypes = [P, I, I, P, P]
        lib.awq_apply_inv_scale.restype = I
        lib.awq_apply_inv_scale.argtypes = [P, P, I, I, P, P]
        lib.awq_pack.restype = I
        lib.awq_pack.argtypes = [P, P, I, I, I, P, P, P, P]
        lib.awq_packed3_sizes.restype = I
        lib.awq_packed3_sizes.argtypes = [I, I, I, ctypes.POINTER(Z), ctypes.POINTER(Z), ctypes.POINTER(Z)]
        lib.awq_pack3.restype = I
        lib.awq_pack3.argtypes = [P, P, I, I, I, P, P, P, P]
        lib.w3a16_gemv.restype = I
        lib.w3a16_gemv.argtypes = [P, P, P, P, P, I, I, I, I, P, Z, P]
        lib.awq_pack_bits.restype = I
        lib.awq_pack_bits.argtypes = [P, P, I, I, I, I, P, P, P, P]
        lib.gptq_quantize.restype = I
        lib.gptq_quantize.argtypes = [P, P, I, I, I, I, ctypes.c_double, P, P, P, P, Z, P]
        lib.gptq_workspace_bytes.restype = Z
        lib.gptq_workspace_bytes.argtypes = [I, I, I, I]
        lib.awq_search_scale.restype = I
        lib.awq_search_scale.argtypes = [P, P, I, I, I, I, I, P, P, P, P, Z, P]
        lib.awq_search_workspace_bytes.restype = Z
        lib.awq_search_workspace_bytes.argtypes = [I, I, I, I, I]
        lib.awq_pack_gate_up.restype = I
        lib.awq_pack_gate_up.argtypes = [P, P, P, I, I, I, P, P, P, P]
        for name in ("w4a16_gemv", "w4a16_gemm", "w4a16_linear", "w4a16_gate_up_silu"):
            fn = getattr(lib, name)
            fn.restype = I
            fn.argtypes = [P, P, P, P, P, I, I, I, I, P, Z, P]
        lib.w4a16_gemv_s.restype = I
        lib.w4a16_gemv_s.argtypes = [P, P, P, P, P, P, I, I, I, I, P, Z, P]
        lib.w4a16_gemv_noalloc.restype = I
        lib.w4a16_gemv_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, P]
        lib.w4a16_linear_pf.restype = I
        lib.w4a16_linear_pf.argtypes = [P, P, P, P, P, I, I, I, I, P, Z, P, Z, P]
        lib.awq_selftest_wait_timeout.restype = I
        lib.awq_selftest_wait_timeout.argtypes = [I, P, P]
        lib.w4a16_gemv_max_m.restype = I
        lib.w4a16_gemv_max_m.argtypes = [I, I]
        lib.w4a16_workspace_bytes.restype = Z
        lib.w4a16_workspace_bytes.argtypes = [I, I, I, I, I]
        lib.awq_last_device_status.restype = I
        lib.awq_last_device_status.argtypes = [P]
        F = ctypes.c_float
        for name, restype, argtypes in (
                ("fp8_scale_bytes", Z, [I, I]),
                ("fp8_quantize", I, [P, I, I, I, P, P, P]),
                ("w8a8_gemm", I, [P, P, P, P, P, I, I, I, I, P]),
                ("w8a8_linear", I, [P, I, P, P, P, I, I, I, P, Z, P]),
                ("w8a8_workspace_bytes", Z, [I, I, I]),
                ("moe_route", I, [P, I, P, I, I, I, I, I, I, I, F, P, P, P]),
                ("w8a8_moe", I, [P, I, P, P, P, P, P, P, P, I, I, I, I, I, I, P, Z, P]),
                ("w8a8_moe_workspace_bytes", Z, [I, I, I, I, I, I])):
            getattr(lib, name).restype = restype
            getattr(lib, name).argtypes = argtypes
        _lib = lib
        return lib


_calls = None


def _foreign(fn):
    """A ctypes function that refuses what csrc/calls.c refuses (ctypes alone cuts whole numbers to their type)."""
    kinds = fn.argtypes

    def call(*args):
        if len(args) != len(kinds):
            raise TypeError(f"{len(kinds)} arguments expected, {len(args)} given")
        values = []
        for a, kind in zip(args, kinds):
            if kind is ctypes.c_float:
                a = float(a) if hasattr(a, "__float__") else operator.index(a)
            elif a is not None or kind is not ctypes.c_void_p:
                a = operator.index(a)
                if kind(a).value != (a or (None if kind is ctypes.c_void_p else 0)):
                    raise OverflowError(f"{a} does not fit its type")
            values.append(a)
        return fn(*values)
    return call


class _ForeignCalls:
    def __init__(self, lib: ctypes.CDLL):
        for name in ("fp8_quantize", "w8a8_gemm", "w8a8_linear", "moe_route", "w8a8_moe"):
            setattr(self, name, _foreign(getattr(lib, name)))


def calls():
    """The 8-bit operators' entry points: the CPython module (csrc/calls.c) over the same library, or, where it could not be
    built, the library's functions by ctypes, about 1 us slower per call."""
    global _calls
    if _calls is None:
        lib = load()
        if os.path.exists(_build.CALLS_PATH):
            from . import _calls as module
            _calls = module
        else:
            _calls = _ForeignCalls(lib)
    return _calls


def check(status: int, where: str) -> None:
    if status != 0:
        raise AwqError(where, status)
