"""8-bit block-scaled operators -- Python binding: the quantizer, the linear layer, the expert router, the expert MLP.

An 8-bit matrix is e4m3 codes [..., R, K] and power-of-two scales (e8m0) [..., R, SC], one per row and block of 128
columns, SC = ceil(K / 128) rounded up to a multiple of 4.  Weights of E experts are one matrix with a leading dimension.
Scratch comes from torch's allocator in each call (it follows the current stream and may be captured); nothing is kept.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Union

import torch

from . import _lib
from ._lib import AwqError

_DTYPES = {torch.float16: 1, torch.bfloat16: 2, torch.float32: 3}
_SCORES = {"softmax": 1, "sigmoid": 2}
_CODES, _SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu


class Fp8Matrix(NamedTuple):
    codes: torch.Tensor    # float8_e4m3fn [..., R, K]
    scales: torch.Tensor   # float8_e8m0fnu [..., R, SC]


class Routing(NamedTuple):
    ids: torch.Tensor      # int32 [M, topk]
    weights: torch.Tensor  # float32 [M, topk]


def fp8_scale_cols(K: int) -> int:
    """Scales per row of an 8-bit matrix of K columns (those past the last block are 1 and not read)."""
    return (K + 511) // 512 * 4


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _call(fn: str, device: torch.device, *args) -> None:
    """Calls the library with `device` current (it launches on the current device)."""
    f = getattr(_lib.load(), fn)
    if device.index == torch.cuda.current_device():
        _lib.check(f(*args), fn)
    else:
        with torch.cuda.device(device):
            _lib.check(f(*args), fn)


def _need(t: torch.Tensor, name: str, dtypes, ndim: int, device: Optional[torch.device] = None) -> None:
    if not t.is_cuda or t.dtype not in dtypes or t.dim() != ndim or not t.is_contiguous():
        kinds = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be a contiguous CUDA {kinds} tensor of {ndim} dimensions")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _need_matrix(m: Fp8Matrix, name: str, ndim: int, device: torch.device) -> None:
    _need(m.codes, f"{name}.codes", (_CODES,), ndim, device)
    _need(m.scales, f"{name}.scales", (_SCALES,), ndim, device)
    want = (*m.codes.shape[:-1], fp8_scale_cols(m.codes.shape[-1]))
    if tuple(m.scales.shape) != want:
        raise ValueError(f"{name}.scales has shape {tuple(m.scales.shape)}, expected {want}")


def _output(out: Optional[torch.Tensor], shape, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(out, "out", (dtype,), len(shape), device)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    return out


def _scratch(fn: str, need: int, workspace: Optional[torch.Tensor], device: torch.device) -> torch.Tensor:
    if need == 2**64 - 1:
        raise AwqError(fn, 1)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def fp8_quantize(x: torch.Tensor, out: Optional[Fp8Matrix] = None) -> Fp8Matrix:
    """Codes and scales of a float16 or bfloat16 matrix [R, K], or of a stack [E, R, K] of them; K % 16 == 0."""
    if x.dim() not in (2, 3):
        raise ValueError("x must have 2 or 3 dimensions")
    _need(x, "x", (torch.float16, torch.bfloat16), x.dim())
    K = x.shape[-1]
    R = x.shape[0] if x.dim() == 2 else x.shape[0] * x.shape[1]
    dev = x.device
    if out is None:
        out = Fp8Matrix(torch.empty(x.shape, dtype=_CODES, device=dev),
                        torch.empty((*x.shape[:-1], fp8_scale_cols(K)), dtype=_SCALES, device=dev))
    else:
        _need_matrix(out, "out", x.dim(), dev)
        if out.codes.shape != x.shape:
            raise ValueError(f"out has shape {tuple(out.codes.shape)}, expected {tuple(x.shape)}")
    _call("fp8_quantize", dev, x.data_ptr(), _DTYPES[x.dtype], R, K, out.codes.data_ptr(), out.scales.data_ptr(),
          _stream(dev))
    return out


def w8a8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.load().w8a8_workspace_bytes(M, N, K))


def w8a8_linear(x: Union[torch.Tensor, Fp8Matrix], w: Fp8Matrix, out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """y [M, N] = x [M, K] w [N, K]^T.  x is float16 or bfloat16, quantized on the way (y has its type), or already an
    Fp8Matrix (one quantization for several weights; `dtype`, or out's, is y's type, bfloat16 unless given)."""
    if isinstance(x, Fp8Matrix):
        dev = x.codes.device
        _need_matrix(x, "x", 2, dev)
        dtype = dtype or (torch.bfloat16 if out is None else out.dtype)
        if dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"dtype must be float16 or bfloat16, not {dtype}")
        M, K = x.codes.shape
    else:
        _need(x, "x", (torch.float16, torch.bfloat16), 2)
        dev = x.device
        if dtype not in (None, x.dtype):
            raise ValueError(f"dtype {dtype} differs from x's {x.dtype}")
        dtype = x.dtype
        M, K = x.shape
    _need_matrix(w, "w", 2, dev)
    N = w.codes.shape[0]
    if w.codes.shape[1] != K:
        raise ValueError(f"x has K={K}, w has K={w.codes.shape[1]}")
    y = _output(out, (M, N), dtype, dev)
    if isinstance(x, Fp8Matrix):
        _call("w8a8_gemm", dev, x.codes.data_ptr(), x.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(),
              y.data_ptr(), _DTYPES[dtype], M, N, K, _stream(dev))
        return y
    ws = _scratch("w8a8_linear", w8a8_workspace_bytes(M, N, K), workspace, dev)
    _call("w8a8_linear", dev, x.data_ptr(), _DTYPES[dtype], w.codes.data_ptr(), w.scales.data_ptr(), y.data_ptr(), M, N, K,
          ws.data_ptr(), ws.numel() * ws.element_size(), _stream(dev))
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
    ids = torch.empty((M, topk), dtype=torch.int32, device=dev)
    weights = torch.empty((M, topk), dtype=torch.float32, device=dev)
    _call("moe_route", dev, logits.data_ptr(), _DTYPES[logits.dtype], 0 if bias is None else bias.data_ptr(), M, E, topk,
          _SCORES[score], groups, topk_groups, int(renorm), scale, ids.data_ptr(), weights.data_ptr(), _stream(dev))
    return Routing(ids, weights)


def w8a8_moe_workspace_bytes(M: int, E: int, topk: int, K: int, I: int, N: int) -> int:
    return int(_lib.load().w8a8_moe_workspace_bytes(M, E, topk, K, I, N))


def w8a8_moe(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate_up: Fp8Matrix, down: Fp8Matrix,
             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] = sum over a token's slots of weights * down[e] Q(silu(gate[e] x) * up[e] x), e = ids.  gate_up
    [E, 2 I, K] (gate rows first), down [E, N, I]; an id outside 0 .. E - 1 adds nothing."""
    _need(x, "x", (torch.float16, torch.bfloat16), 2)
    dev = x.device
    M, K = x.shape
    _need(ids, "ids", (torch.int32,), 2, dev)
    _need(weights, "weights", (torch.float32,), 2, dev)
    _need_matrix(gate_up, "gate_up", 3, dev)
    _need_matrix(down, "down", 3, dev)
    E, two_i, gk = gate_up.codes.shape
    topk = ids.shape[1]
    if ids.shape[0] != M or weights.shape != ids.shape:
        raise ValueError(f"ids {tuple(ids.shape)} and weights {tuple(weights.shape)} do not match {M} tokens")
    if gk != K or two_i % 2 != 0 or down.codes.shape[0] != E or down.codes.shape[2] * 2 != two_i:
        raise ValueError(f"gate_up {tuple(gate_up.codes.shape)} and down {tuple(down.codes.shape)} do not match x's K={K}")
    N, I = down.codes.shape[1:]
    y = _output(out, (M, N), x.dtype, dev)
    ws = _scratch("w8a8_moe", w8a8_moe_workspace_bytes(M, E, topk, K, I, N), workspace, dev)
    _call("w8a8_moe", dev, x.data_ptr(), _DTYPES[x.dtype], ids.data_ptr(), weights.data_ptr(), gate_up.codes.data_ptr(),
          gate_up.scales.data_ptr(), down.codes.data_ptr(), down.scales.data_ptr(), y.data_ptr(), M, E, topk, K, I, N,
          ws.data_ptr(), ws.numel() * ws.element_size(), _stream(dev))
    return y
