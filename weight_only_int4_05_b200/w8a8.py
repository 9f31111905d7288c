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
_LOGITS = tuple(_DTYPES)
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
# The raw forms of current_device() and current_stream(): these calls take microseconds, and building a Stream is one of them.
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


class Fp8Matrix(NamedTuple):
    codes: torch.Tensor    # float8_e4m3fn [..., R, K]
    scales: torch.Tensor   # float8_e8m0fnu [..., R, SC]


class Routing(NamedTuple):
    ids: torch.Tensor      # int32 [M, topk]
    weights: torch.Tensor  # float32 [M, topk]


def fp8_scale_cols(K: int) -> int:
    """Scales per row of an 8-bit matrix of K columns (those past the last block are 1 and not read)."""
    return (K + 511) // 512 * 4


def _need(t: torch.Tensor, name: str, dtypes, ndim: int) -> None:
    if t.dtype not in dtypes or not t.is_cuda or t.dim() != ndim or not t.is_contiguous():
        kinds = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be a contiguous CUDA {kinds} tensor of {ndim} dimensions")


def _need_on(t: torch.Tensor, name: str, dtypes, ndim: int, device: torch.device) -> None:
    _need(t, name, dtypes, ndim)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _need_matrix(m: Fp8Matrix, name: str, ndim: int, device: torch.device):
    """Checks an 8-bit matrix and returns the shape of its codes."""
    codes, scales = m
    shape, of = codes.shape, scales.shape
    if (codes.dtype is not _E4M3 or scales.dtype is not _E8M0 or codes.device != device or scales.device != device
            or not codes.is_cuda or len(shape) != ndim or len(of) != ndim or not codes.is_contiguous()
            or not scales.is_contiguous() or of[-1] != fp8_scale_cols(shape[-1]) or of[:-1] != shape[:-1]):
        _need_on(codes, f"{name}.codes", (_E4M3,), ndim, device)
        _need_on(scales, f"{name}.scales", (_E8M0,), ndim, device)
        raise ValueError(f"{name}.scales has shape {tuple(of)}, expected {(*shape[:-1], fp8_scale_cols(shape[-1]))}")
    return shape


def _output(out: Optional[torch.Tensor], M: int, N: int, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    if out is None:
        return torch.empty(M, N, dtype=dtype, device=device)
    _need_on(out, "out", (dtype,), 2, device)
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


# Each call launches on the current device: one whose tensors are on another device makes that one current first.


def fp8_quantize(x: torch.Tensor, out: Optional[Fp8Matrix] = None) -> Fp8Matrix:
    """Codes and scales of a float16 or bfloat16 matrix [R, K], or of a stack [E, R, K] of them; K % 16 == 0."""
    shape = x.shape
    if len(shape) == 2:
        R, K = shape
    elif len(shape) == 3:
        R, K = shape[0] * shape[1], shape[2]
    else:
        raise ValueError("x must have 2 or 3 dimensions")
    _need(x, "x", _HALF, len(shape))
    dev = x.device
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return fp8_quantize(x, out)
    if out is None:
        out = Fp8Matrix(torch.empty_like(x, dtype=_E4M3),
                        torch.empty(*shape[:-1], fp8_scale_cols(K), dtype=_E8M0, device=dev))
    elif _need_matrix(out, "out", len(shape), dev) != shape:
        raise ValueError(f"out has shape {tuple(out.codes.shape)}, expected {tuple(shape)}")
    status = _lib.calls().fp8_quantize(x.data_ptr(), _DTYPES[x.dtype], R, K, out[0].data_ptr(), out[1].data_ptr(),
                                       _current_stream(dev.index))
    if status:
        _lib.check(status, "fp8_quantize")
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
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return w8a8_linear(x, w, out, workspace, dtype)
    N, wk = _need_matrix(w, "w", 2, dev)
    if wk != K:
        raise ValueError(f"x has K={K}, w has K={wk}")
    y = _output(out, M, N, dtype, dev)
    lib = _lib.calls()
    if quantized:
        status = lib.w8a8_gemm(x.codes.data_ptr(), x.scales.data_ptr(), w[0].data_ptr(), w[1].data_ptr(), y.data_ptr(),
                               _DTYPES[dtype], M, N, K, _current_stream(dev.index))
    else:
        ws, at, size = _scratch("w8a8_linear", w8a8_workspace_bytes(M, N, K), workspace, dev)
        status = lib.w8a8_linear(x.data_ptr(), _DTYPES[dtype], w[0].data_ptr(), w[1].data_ptr(), y.data_ptr(), M, N, K, at,
                                 size, _current_stream(dev.index))
    if status:
        _lib.check(status, "w8a8_linear")
    return y


def moe_route(logits: torch.Tensor, topk: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
              groups: int = 1, topk_groups: int = 1, renorm: bool = False, scale: float = 1.0) -> Routing:
    """The topk experts of each token from logits [M, E] (float32, float16 or bfloat16) and their weights.  bias
    [E] float32 counts in the choice only; with groups > 1 the choice is among the topk_groups best groups."""
    _need(logits, "logits", _LOGITS, 2)
    dev = logits.device
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return moe_route(logits, topk, score, bias, groups, topk_groups, renorm, scale)
    M, E = logits.shape
    kind = _SCORES.get(score)
    if kind is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    at = None
    if bias is not None:
        _need_on(bias, "bias", (torch.float32,), 1, dev)
        if bias.shape[0] != E:
            raise ValueError(f"bias has shape {tuple(bias.shape)}, expected ({E},)")
        at = bias.data_ptr()
    if topk < 1 or topk > 32:
        raise AwqError("moe_route", 1)
    ids = torch.empty(M, topk, dtype=torch.int32, device=dev)
    weights = torch.empty(M, topk, dtype=torch.float32, device=dev)
    status = _lib.calls().moe_route(logits.data_ptr(), _DTYPES[logits.dtype], at, M, E, topk, kind, groups, topk_groups,
                                    1 if renorm else 0, scale, ids.data_ptr(), weights.data_ptr(),
                                    _current_stream(dev.index))
    if status:
        _lib.check(status, "moe_route")
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
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return w8a8_moe(x, ids, weights, gate_up, down, out, workspace)
    M, K = x.shape
    _need_on(ids, "ids", (torch.int32,), 2, dev)
    _need_on(weights, "weights", (torch.float32,), 2, dev)
    E, two_i, gk = _need_matrix(gate_up, "gate_up", 3, dev)
    de, N, I = _need_matrix(down, "down", 3, dev)
    rows, topk = ids.shape
    if rows != M or weights.shape != ids.shape:
        raise ValueError(f"ids {tuple(ids.shape)} and weights {tuple(weights.shape)} do not match {M} tokens")
    if gk != K or de != E or 2 * I != two_i:
        raise ValueError(f"gate_up {tuple(gate_up.codes.shape)} and down {tuple(down.codes.shape)} do not match x's K={K}")
    y = _output(out, M, N, x.dtype, dev)
    ws, at, size = _scratch("w8a8_moe", w8a8_moe_workspace_bytes(M, E, topk, K, I, N), workspace, dev)
    status = _lib.calls().w8a8_moe(x.data_ptr(), _DTYPES[x.dtype], ids.data_ptr(), weights.data_ptr(), gate_up[0].data_ptr(),
                                  gate_up[1].data_ptr(), down[0].data_ptr(), down[1].data_ptr(), y.data_ptr(), M, E, topk, K,
                                  I, N, at, size, _current_stream(dev.index))
    if status:
        _lib.check(status, "w8a8_moe")
    return y
