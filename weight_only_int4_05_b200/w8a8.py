"""8-bit block-scaled operators -- Python binding: the quantizer, the linear layer, the expert router, the expert MLP.

An 8-bit matrix is e4m3 codes [..., R, K] and power-of-two scales (e8m0) [..., R, SC], one per row and block of 128
columns, SC = ceil(K / 128) rounded up to a multiple of 4.  Weights of E experts are one matrix with a leading dimension.
Scratch comes from torch's allocator in each call (it follows the current stream and may be captured); nothing is kept.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Union

import torch

from . import _lib
from ._lib import AwqError

_DTYPES = {torch.float16: 1, torch.bfloat16: 2, torch.float32: 3}
_SCORES = {"softmax": 1, "sigmoid": 2}
_HALF = (torch.float16, torch.bfloat16)
_CODES, _SCALES = (torch.float8_e4m3fn,), (torch.float8_e8m0fnu,)


class Fp8Matrix(NamedTuple):
    codes: torch.Tensor    # float8_e4m3fn [..., R, K]
    scales: torch.Tensor   # float8_e8m0fnu [..., R, SC]


class Routing(NamedTuple):
    ids: torch.Tensor      # int32 [M, topk]
    weights: torch.Tensor  # float32 [M, topk]


def fp8_scale_cols(K: int) -> int:
    """Scales per row of an 8-bit matrix of K columns (those past the last block are 1 and not read)."""
    return (K + 511) // 512 * 4


def _library(device: torch.device):
    """The library and the raw handle of the device's current stream; these calls take microseconds, so the handle is
    read without building a Stream object."""
    return _lib.load(), torch._C._cuda_getCurrentRawStream(device.index)


def _run(fn: str, f, device: torch.device, args) -> None:
    """Calls the library with `device` current (it launches on the current device)."""
    if device.index == torch._C._cuda_getDevice():
        status = f(*args)
    else:
        with torch.cuda.device(device):
            status = f(*args)
    if status:
        _lib.check(status, fn)


def _need(t: torch.Tensor, name: str, dtypes, ndim: int, device: Optional[torch.device] = None) -> None:
    if t.dtype not in dtypes or not t.is_cuda or t.dim() != ndim or not t.is_contiguous():
        kinds = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be a contiguous CUDA {kinds} tensor of {ndim} dimensions")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _need_matrix(m: Fp8Matrix, name: str, ndim: int, device: torch.device):
    """Checks an 8-bit matrix and returns the shape of its codes."""
    codes, scales = m
    _need(codes, f"{name}.codes", _CODES, ndim, device)
    _need(scales, f"{name}.scales", _SCALES, ndim, device)
    shape = codes.shape
    if scales.shape[-1] != fp8_scale_cols(shape[-1]) or scales.shape[:-1] != shape[:-1]:
        raise ValueError(f"{name}.scales has shape {tuple(scales.shape)}, expected "
                         f"{(*shape[:-1], fp8_scale_cols(shape[-1]))}")
    return shape


def _output(out: Optional[torch.Tensor], M: int, N: int, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    if out is None:
        return torch.empty(M, N, dtype=dtype, device=device)
    _need(out, "out", (dtype,), 2, device)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(M, N)}")
    return out


def _scratch(fn: str, need: int, workspace: Optional[torch.Tensor], device: torch.device):
    """The scratch tensor of a call, its address and bytes."""
    if need == 2**64 - 1:
        raise AwqError(fn, 1)
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.nbytes


def fp8_quantize(x: torch.Tensor, out: Optional[Fp8Matrix] = None) -> Fp8Matrix:
    """Codes and scales of a float16 or bfloat16 matrix [R, K], or of a stack [E, R, K] of them; K % 16 == 0."""
    shape = x.shape
    if len(shape) not in (2, 3):
        raise ValueError("x must have 2 or 3 dimensions")
    _need(x, "x", _HALF, len(shape))
    K = shape[-1]
    R = shape[0] if len(shape) == 2 else shape[0] * shape[1]
    dev = x.device
    if out is None:
        out = Fp8Matrix(torch.empty_like(x, dtype=_CODES[0]),
                        torch.empty(*shape[:-1], fp8_scale_cols(K), dtype=_SCALES[0], device=dev))
    elif _need_matrix(out, "out", len(shape), dev) != shape:
        raise ValueError(f"out has shape {tuple(out.codes.shape)}, expected {tuple(shape)}")
    lib, stream = _library(dev)
    _run("fp8_quantize", lib.fp8_quantize, dev, (x.data_ptr(), _DTYPES[x.dtype], R, K, out.codes.data_ptr(),
                                                 out.scales.data_ptr(), stream))
    return out


@functools.lru_cache(maxsize=4096)
def w8a8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.load().w8a8_workspace_bytes(M, N, K))


def w8a8_linear(x: Union[torch.Tensor, Fp8Matrix], w: Fp8Matrix, out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """y [M, N] = x [M, K] w [N, K]^T.  x is float16 or bfloat16, quantized on the way (y has its type), or already an
    Fp8Matrix (one quantization for several weights; `dtype`, or out's, is y's type, bfloat16 unless given)."""
    quantized = isinstance(x, Fp8Matrix)
    if quantized:
        dev = x.codes.device
        M, K = _need_matrix(x, "x", 2, dev)
        dtype = dtype or (torch.bfloat16 if out is None else out.dtype)
        if dtype not in _HALF:
            raise ValueError(f"dtype must be float16 or bfloat16, not {dtype}")
    else:
        _need(x, "x", _HALF, 2)
        dev = x.device
        if dtype is not None and dtype != x.dtype:
            raise ValueError(f"dtype {dtype} differs from x's {x.dtype}")
        dtype = x.dtype
        M, K = x.shape
    N, wk = _need_matrix(w, "w", 2, dev)
    if wk != K:
        raise ValueError(f"x has K={K}, w has K={wk}")
    y = _output(out, M, N, dtype, dev)
    lib, stream = _library(dev)
    if quantized:
        _run("w8a8_gemm", lib.w8a8_gemm, dev, (x.codes.data_ptr(), x.scales.data_ptr(), w.codes.data_ptr(),
                                               w.scales.data_ptr(), y.data_ptr(), _DTYPES[dtype], M, N, K, stream))
        return y
    ws, at, size = _scratch("w8a8_linear", w8a8_workspace_bytes(M, N, K), workspace, dev)
    _run("w8a8_linear", lib.w8a8_linear, dev, (x.data_ptr(), _DTYPES[dtype], w.codes.data_ptr(), w.scales.data_ptr(),
                                               y.data_ptr(), M, N, K, at, size, stream))
    return y


def moe_route(logits: torch.Tensor, topk: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
              groups: int = 1, topk_groups: int = 1, renorm: bool = False, scale: float = 1.0) -> Routing:
    """The topk experts of each token from logits [M, E] (float32, float16 or bfloat16) and their weights.  bias
    [E] float32 counts in the choice only; with groups > 1 the choice is among the topk_groups best groups."""
    _need(logits, "logits", tuple(_DTYPES), 2)
    dev = logits.device
    M, E = logits.shape
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    if bias is not None:
        _need(bias, "bias", (torch.float32,), 1, dev)
        if bias.shape[0] != E:
            raise ValueError(f"bias has shape {tuple(bias.shape)}, expected ({E},)")
    if topk < 1 or topk > 32:
        raise AwqError("moe_route", 1)
    ids = torch.empty(M, topk, dtype=torch.int32, device=dev)
    weights = torch.empty(M, topk, dtype=torch.float32, device=dev)
    lib, stream = _library(dev)
    _run("moe_route", lib.moe_route, dev, (
        logits.data_ptr(), _DTYPES[logits.dtype], None if bias is None else bias.data_ptr(), M, E, topk, _SCORES[score],
        groups, topk_groups, bool(renorm), scale, ids.data_ptr(), weights.data_ptr(), stream))
    return Routing(ids, weights)


@functools.lru_cache(maxsize=4096)
def w8a8_moe_workspace_bytes(M: int, E: int, topk: int, K: int, I: int, N: int) -> int:
    return int(_lib.load().w8a8_moe_workspace_bytes(M, E, topk, K, I, N))


def w8a8_moe(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate_up: Fp8Matrix, down: Fp8Matrix,
             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] = sum over a token's slots of weights * down[e] Q(silu(gate[e] x) * up[e] x), e = ids.  gate_up
    [E, 2 I, K] (gate rows first), down [E, N, I]; an id outside 0 .. E - 1 adds nothing."""
    _need(x, "x", _HALF, 2)
    dev = x.device
    M, K = x.shape
    _need(ids, "ids", (torch.int32,), 2, dev)
    _need(weights, "weights", (torch.float32,), 2, dev)
    E, two_i, gk = _need_matrix(gate_up, "gate_up", 3, dev)
    de, N, I = _need_matrix(down, "down", 3, dev)
    topk = ids.shape[1]
    if ids.shape[0] != M or weights.shape != ids.shape:
        raise ValueError(f"ids {tuple(ids.shape)} and weights {tuple(weights.shape)} do not match {M} tokens")
    if gk != K or de != E or 2 * I != two_i:
        raise ValueError(f"gate_up {tuple(gate_up.codes.shape)} and down {tuple(down.codes.shape)} do not match x's K={K}")
    y = _output(out, M, N, x.dtype, dev)
    ws, at, size = _scratch("w8a8_moe", w8a8_moe_workspace_bytes(M, E, topk, K, I, N), workspace, dev)
    lib, stream = _library(dev)
    _run("w8a8_moe", lib.w8a8_moe, dev, (
        x.data_ptr(), _DTYPES[x.dtype], ids.data_ptr(), weights.data_ptr(), gate_up.codes.data_ptr(),
        gate_up.scales.data_ptr(), down.codes.data_ptr(), down.scales.data_ptr(), y.data_ptr(), M, E, topk, K, I, N,
        at, size, stream))
    return y
