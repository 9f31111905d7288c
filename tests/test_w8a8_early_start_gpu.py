"""Products behind a kernel that lets them start at once and then runs longer than a bounded wait (2 s): they wait for it without
counting its time."""
import pytest
import torch

import fp8_device
import weight_only_int4_05_b200 as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["one token", "16 tokens", "40 tokens", "experts"])
def test_behind_a_kernel_of_two_and_a_half_seconds(form):
    g = torch.Generator("cuda").manual_seed(3)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=g).half()  # noqa: E731
    if form == "experts":
        x, gu, dn = rand(24, 2048), W.fp8_quantize(rand(4, 512, 2048) * 0.02), W.fp8_quantize(rand(4, 512, 256) * 0.02)
        ids = torch.randint(0, 4, (24, 2), device="cuda", generator=g, dtype=torch.int32)
        weights = torch.ones(24, 2, device="cuda")
        call = lambda: W.w8a8_moe(x, ids, weights, gu, dn)  # noqa: E731
    else:  # K of 8 and 12 words of scales, and tiles of 128 outputs
        M, N, K = {"one token": (1, 512, 4096), "16 tokens": (16, 40000, 6144), "40 tokens": (40, 512, 4096)}[form]
        x, w = rand(M, K), W.fp8_quantize(rand(N, K) * 0.02)
        call = lambda: W.w8a8_linear(x, w)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    assert fp8_device.load().signal_then_run(2_500_000_000, torch.cuda.current_stream().cuda_stream) == 0
    got = call()
    torch.cuda.synchronize()
    assert W.awq_last_device_status() == 0
    assert torch.equal(got, want)
