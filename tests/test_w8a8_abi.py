"""Argument checks of the 8-bit operators that need no GPU: every refusal happens on the host before a launch."""
import ctypes

import pytest
import torch

import weight_only_int4_05_b200 as W
from weight_only_int4_05_b200 import _lib, build as libbuild

P, F, Z = ctypes.c_void_p, ctypes.c_void_p(0x10000), 2**64 - 1
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return _lib.load()


def test_sizes(L):
    assert L.fp8_scale_bytes(3, 16) == 12 and L.fp8_scale_bytes(3, 512) == 12 and L.fp8_scale_bytes(3, 528) == 24
    assert L.fp8_scale_bytes(0, 512) == Z and L.fp8_scale_bytes(3, 24) == Z and L.fp8_scale_bytes(3, 0) == Z
    assert W.fp8_scale_cols(16) == 4 and W.fp8_scale_cols(4096) == 32 and W.fp8_scale_cols(4112) == 36
    assert L.w8a8_workspace_bytes(17, 8, 512) >= 17 * (512 + 4)
    assert L.w8a8_workspace_bytes(16, 8, 512) == 0  # the product quantizes few tokens itself
    assert L.w8a8_workspace_bytes(0, 8, 512) == Z and L.w8a8_workspace_bytes(1, 8, 520) == Z
    assert L.w8a8_moe_workspace_bytes(4, 8, 2, 512, 256, 512) >= 8 * (512 + 256 + 4 * 512)
    for bad in ((0, 8, 2, 512, 256, 512), (4, 0, 2, 512, 256, 512), (4, 1025, 2, 512, 256, 512),
                (4, 8, 0, 512, 256, 512), (4, 8, 33, 512, 256, 512), (4, 8, 2, 500, 256, 512),
                (4, 8, 2, 512, 250, 512), (4, 8, 2, 512, 256, 0), (1 << 22, 8, 8, 512, 256, 512),
                (4, 1024, 2, 512, (1 << 19) + 16, 512), (4, 1024, 2, 512, 256, (1 << 20) + 1)):
        assert L.w8a8_moe_workspace_bytes(*bad) == Z, bad


def test_quantize_checks(L):
    assert L.fp8_quantize(F, 3, 4, 512, F, F, None) == 2
    assert L.fp8_quantize(F, 0, 4, 512, F, F, None) == 2
    assert L.fp8_quantize(F, 1, 0, 512, F, F, None) == 1
    assert L.fp8_quantize(F, 1, (1 << 30) + 1, 16, F, F, None) == 1
    assert L.fp8_quantize(F, 1, 4, 504, F, F, None) == 1
    assert L.fp8_quantize(None, 1, 4, 512, F, F, None) == 1
    assert L.fp8_quantize(F, 1, 4, 512, F, None, None) == 1
    assert L.fp8_quantize(ODD, 1, 4, 512, F, F, None) == 3
    assert L.fp8_quantize(F, 2, 4, 512, F, ODD, None) == 3


def test_linear_checks(L):
    big = 1 << 40
    lin = lambda x=F, dt=1, wc=F, ws=F, y=F, M=40, N=8, K=512, work=F, n=big: L.w8a8_linear(  # noqa: E731
        x, dt, wc, ws, y, M, N, K, work, n, None)
    assert lin(dt=3) == 2
    assert lin(M=0) == 1 and lin(N=0) == 1 and lin(K=0) == 1 and lin(K=520) == 1 and lin(M=-1) == 1
    assert lin(x=None) == 1 and lin(wc=None) == 1 and lin(ws=None) == 1 and lin(y=None) == 1
    assert lin(x=ODD) == 3 and lin(wc=ODD) == 3 and lin(ws=ODD) == 3 and lin(y=ODD) == 3 and lin(work=ODD) == 3
    assert lin(work=None) == 6 and lin(n=16) == 6
    mm = lambda xc=F, xs=F, dt=1, M=4, N=8, K=512: L.w8a8_gemm(xc, xs, F, F, F, dt, M, N, K, None)  # noqa: E731
    assert mm(dt=3) == 2 and mm(M=0) == 1 and mm(K=8) == 1 and mm(xs=None) == 1 and mm(xs=ODD) == 3 and mm(xc=ODD) == 3


def test_outputs_over_inputs_are_refused(L):
    """Every call here has one pair of arrays that share bytes, its last 16 among them, and is refused before a launch."""
    far = [(i + 1) << 40 for i in range(11)]
    def refused(call, n, i, nbytes, j):  # array j starts in the last 16 bytes of array i
        for at in (far[i], far[i] + nbytes - 16):
            p = far[:n]
            p[j] = at
            assert call([P(v) for v in p]) == 1, (i, j)
    q = lambda p: L.fp8_quantize(p[0], 1, 64, 512, p[1], p[2], None)  # noqa: E731
    refused(q, 3, 0, 64 * 512 * 2, 1), refused(q, 3, 0, 64 * 512 * 2, 2), refused(q, 3, 1, 64 * 512, 2)
    mm = lambda p: L.w8a8_gemm(p[0], p[1], p[2], p[3], p[4], 1, 64, 32, 512, None)  # noqa: E731
    for i, n in ((0, 64 * 512), (1, 64 * 4), (2, 32 * 512), (3, 32 * 4)):
        refused(mm, 5, i, n, 4)
    for M in (4, 64):
        lin = lambda p: L.w8a8_linear(p[0], 1, p[1], p[2], p[3], M, 32, 512, p[4], 1 << 40, None)  # noqa: E731
        for i, n in ((0, M * 512 * 2), (1, 32 * 512), (2, 32 * 4)):
            refused(lin, 5, i, n, 3)
    refused(lin, 5, 0, 64 * 512 * 2, 4), refused(lin, 5, 3, 64 * 32 * 2, 4)
    route = lambda p: L.moe_route(p[0], 3, p[1], 64, 64, 4, 1, 1, 1, 0, ctypes.c_float(1), p[2], p[3], None)  # noqa: E731
    for i, n in ((0, 64 * 64 * 4), (1, 64 * 4)):
        refused(route, 4, i, n, 2), refused(route, 4, i, n, 3)
    refused(route, 4, 2, 64 * 4 * 4, 3)
    moe = lambda p: L.w8a8_moe(p[0], 1, p[1], p[2], p[3], p[4], p[5], p[6], p[7], 64, 8, 2, 512, 256, 128, p[8],  # noqa: E731
                               1 << 40, None)
    refused(moe, 9, 2, 64 * 2 * 4, 7)
    for i, n in ((0, 64 * 512 * 2), (1, 64 * 2 * 4), (2, 64 * 2 * 4), (7, 64 * 128 * 2)):
        refused(moe, 9, i, n, 8)


def test_route_checks(L):
    route = lambda l=F, dt=3, b=None, M=4, E=64, k=4, s=1, g=1, tg=1, sc=1.0, i=F, w=F: L.moe_route(  # noqa: E731
        l, dt, b, M, E, k, s, g, tg, 0, ctypes.c_float(sc), i, w, None)
    assert route(dt=4) == 2 and route(s=0) == 2 and route(s=3) == 2
    assert route(M=0) == 1 and route(E=0) == 1 and route(E=1025) == 1 and route(k=0) == 1
    assert route(k=33) == 1 and route(E=3, k=4) == 1
    assert route(g=0) == 1 and route(g=5, tg=1) == 1 and route(g=64, tg=64) == 1 and route(g=8, tg=9) == 1
    assert route(g=8, tg=0) == 1 and route(g=32, tg=1) == 1          # 4 experts out of 1 group of 2
    assert route(sc=float("nan")) == 1
    assert route(l=None) == 1 and route(i=None) == 1 and route(w=None) == 1
    assert route(l=ODD) == 3 and route(b=ODD) == 3 and route(i=ODD) == 3 and route(w=ODD) == 3


def test_moe_checks(L):
    big = 1 << 40
    def moe(x=F, dt=1, ids=F, w=F, gc=F, gs=F, dc=F, ds=F, y=F, M=4, E=8, k=2, K=512, I=256, N=512, work=F, n=big):
        return L.w8a8_moe(x, dt, ids, w, gc, gs, dc, ds, y, M, E, k, K, I, N, work, n, None)
    assert moe(dt=3) == 2
    assert moe(M=0) == 1 and moe(E=0) == 1 and moe(k=0) == 1 and moe(K=8) == 1 and moe(I=24) == 1 and moe(N=0) == 1
    for name in ("x", "ids", "w", "gc", "gs", "dc", "ds", "y"):
        assert moe(**{name: None}) == 1, name
        assert moe(**{name: ODD}) == 3, name
    assert moe(work=None) == 6 and moe(n=100) == 6 and moe(work=ODD) == 3


def test_python_refusals_on_the_host():
    x = torch.zeros(4, 512, dtype=torch.float16)
    m = W.Fp8Matrix(torch.zeros(8, 512).to(torch.float8_e4m3fn), torch.zeros(8, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu))
    for call in (lambda: W.fp8_quantize(x), lambda: W.fp8_quantize(x[0]), lambda: W.w8a8_linear(x, m),
                 lambda: W.w8a8_linear(m, m), lambda: W.moe_route(x, 4),
                 lambda: W.w8a8_moe(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), m, m)):
        with pytest.raises(ValueError):
            call()


def test_calls_module_refuses_like_the_library(L):
    """The CPython functions pass every argument on: the library's refusals come back, and arguments of another kind are
    errors before the call."""
    C, at = _lib.calls(), 0x10000
    assert C.fp8_quantize(at, 3, 4, 512, at, at, None) == 2 and C.fp8_quantize(at, 1, 4, 504, at, at, 0) == 1
    assert C.fp8_quantize(at, 1, 4, 512, at, at + 8, None) == 3
    assert C.w8a8_gemm(at, at, at, at, at, 3, 4, 8, 512, None) == 2 and C.w8a8_gemm(at, None, at, at, at, 1, 4, 8, 512, None) == 1
    assert C.w8a8_linear(at, 1, at, at, at, 400, 8192, 4096, None, 0, None) == 6
    assert C.w8a8_linear(at, 1, at, at, at, 400, 8192, 4096, at, 16, None) == 6
    assert C.w8a8_linear(at, 1, at, at, at, 4, 512, 512, None, 0, None) == 1  # y over x
    assert C.moe_route(at, 3, None, 4, 64, 4, 3, 1, 1, 0, 1.0, at, at, None) == 2
    assert C.moe_route(at, 3, None, 4, 64, 4, 1, 1, 1, 0, float("nan"), at, at, None) == 1
    assert C.moe_route(at, 3, None, 4, 64, 4, 1, 1, 1, 0, 1, at, at + 8, None) == 3
    assert C.w8a8_moe(at, 3, at, at, at, at, at, at, at, 4, 8, 2, 512, 256, 512, at, 1 << 40, None) == 2
    assert C.w8a8_moe(at, 1, at, at, at, at, at, at, at, 4, 8, 2, 512, 250, 512, at, 1 << 40, None) == 1
    assert C.w8a8_moe(at, 1, at, at, at, at, at, at, at, 4, 8, 2, 512, 256, 512, at, 100, None) == 6
    for bad in ((at, 1, 4, 512, at, at), (at, 1, 1 << 40, 512, at, at, None), (at, 1, "4", 512, at, at, None),
                (at, 1, 4.5, 512, at, at, None), ("x", 1, 4, 512, at, at, None)):
        with pytest.raises((TypeError, OverflowError)):
            C.fp8_quantize(*bad)
