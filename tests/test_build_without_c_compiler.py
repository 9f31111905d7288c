"""Where no C compiler (or no Python.h) is found, the library is built all the same and the 8-bit operators' calls go through
ctypes, with the same refusals (no GPU needed)."""
import shutil

import pytest

from weight_only_int4_05_b200 import _lib, build as libbuild


@pytest.fixture
def bare(monkeypatch, tmp_path):
    """A built library, no CPython module beside it, and no C compiler."""
    libbuild.build()
    which = shutil.which
    monkeypatch.setattr(libbuild, "CALLS_PATH", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(libbuild.shutil, "which", lambda c: None if c in ("gcc", "cc") else which(c))
    monkeypatch.delenv("CC", raising=False)
    monkeypatch.setattr(_lib, "_calls", None)


def test_build_succeeds_and_says_so(bare):
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert libbuild.build() == libbuild.LIB_PATH


def test_build_succeeds_without_python_headers(bare, monkeypatch, tmp_path):
    cc = tmp_path / "cc"
    cc.write_text("#!/bin/sh\necho 'Python.h: No such file' >&2\nexit 1\n")
    cc.chmod(0o755)
    monkeypatch.setenv("CC", str(cc))
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert libbuild.build() == libbuild.LIB_PATH


def test_a_module_of_an_older_build_is_not_left_behind(bare, tmp_path):
    (tmp_path / "_calls.so").write_bytes(b"old")
    with pytest.warns(RuntimeWarning):
        libbuild.build(force=False)
        libbuild._build_calls()
    assert not (tmp_path / "_calls.so").exists()


def test_calls_refuse_like_the_module(bare):
    C, at = _lib.calls(), 0x10000
    assert C.fp8_quantize(at, 3, 4, 512, at, at, None) == 2 and C.fp8_quantize(at, 1, 4, 504, at, at, 0) == 1
    assert C.w8a8_gemm(at, None, at, at, at, 1, 4, 8, 512, None) == 1
    assert C.w8a8_linear(at, 1, at, at, at, 400, 8192, 4096, at, 16, None) == 6
    assert C.moe_route(at, 3, None, 4, 64, 4, 1, 1, 1, 0, float("nan"), at, at, None) == 1
    assert C.moe_route(at, 3, None, 4, 64, 4, 1, 1, 1, 0, 1, at, at + 8, None) == 3
    assert C.w8a8_moe(at, 1, at, at, at, at, at, at, at, 4, 8, 2, 512, 256, 512, at, 100, None) == 6
    for bad in ((at, 1, 4, 512, at, at), (at, 1, 1 << 40, 512, at, at, None), (at, 1, "4", 512, at, at, None),
                (at, 1, 4.5, 512, at, at, None), ("x", 1, 4, 512, at, at, None), (at, 1, 4, 512, at, at, 1.5)):
        with pytest.raises((TypeError, OverflowError)):
            C.fp8_quantize(*bad)
    for scale in ("1", None):
        with pytest.raises(TypeError):
            C.moe_route(at, 3, None, 4, 64, 65, 1, 1, 1, 0, scale, at, at, None)
    for size in (-1, 1 << 64, None):
        with pytest.raises((TypeError, OverflowError)):
            C.w8a8_linear(at, 1, at, at, at, 400, 8192, 4096, at, size, None)


@pytest.mark.gpu
def test_operators_through_ctypes_give_the_same(monkeypatch):
    import torch

    import weight_only_int4_05_b200 as W
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(24, 256, device="cuda", generator=g).half()
    gu, dn = torch.randn(4, 128, 256, device="cuda", generator=g).half(), torch.randn(4, 256, 64, device="cuda", generator=g).half()

    def outputs():
        qx, qg, qd = W.fp8_quantize(x), W.fp8_quantize(gu), W.fp8_quantize(dn)
        head = W.Fp8Matrix(qg.codes[0], qg.scales[0])
        r = W.moe_route(W.w8a8_linear(x, head), 2, renorm=True, scale=1.5)
        ids = r.ids % 4
        return [qx.codes.view(torch.uint8), qx.scales.view(torch.uint8), W.w8a8_linear(qx, head), r.ids, r.weights,
                W.w8a8_moe(x, ids, r.weights, qg, qd)]
    module = outputs()
    assert not isinstance(_lib.calls(), _lib._ForeignCalls)
    monkeypatch.setattr(_lib, "_calls", _lib._ForeignCalls(_lib.load()))
    assert all(torch.equal(a, b) for a, b in zip(module, outputs()))
    assert W.awq_last_device_status() == 0
