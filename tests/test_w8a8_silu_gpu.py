"""silu over the whole range of 32-bit values, and experts whose gates reach its ends."""
import numpy as np
import pytest
import torch

import fp8_device
import weight_only_int4_05_b200 as W

pytestmark = pytest.mark.gpu


def test_silu_against_64_bits():
    """The exponential is off by 2^-22 (its instruction) and 2^-24 (the correction's rounding), 1 + e by 2^-24, the quotient by 2
    units in the last place, 2^-22: 2^-21 + 2^-23 of the value together.  Below 2^-119 the value may be 0."""
    rng = np.random.default_rng(1)
    far = np.exp2(rng.uniform(-149, 128, 400000))
    a = np.r_[far, -far, rng.uniform(-110, 110, 1000000), rng.normal(size=200000), 0.0, -0.0].astype(np.float32)
    a = a[np.isfinite(a)]
    x = torch.from_numpy(a).cuda()
    y = torch.empty_like(x)
    assert fp8_device.load().silu_of(x.data_ptr(), y.data_ptr(), len(a), torch.cuda.current_stream().cuda_stream) == 0
    with np.errstate(over="ignore"):
        want = a.astype(np.float64) / (1.0 + np.exp(-a.astype(np.float64)))
    off = np.abs(y.double().cpu().numpy() - want) - ((2.0 ** -21 + 2.0 ** -23) * np.abs(want) + 2.0 ** -119)
    assert not np.isnan(off).any() and off.max() <= 0, (a[off.argmax()], off.max())


def test_silu_at_its_ends():
    big = float(np.finfo(np.float32).max)
    a = [2.3e38, 2.36e38, 2.4e38, big, float("inf"), -2.3e38, -2.4e38, -big, -float("inf"), float("nan")]
    x = torch.tensor(a, device="cuda")
    y = torch.empty_like(x)
    assert fp8_device.load().silu_of(x.data_ptr(), y.data_ptr(), len(a), torch.cuda.current_stream().cuda_stream) == 0
    y = y.cpu()
    assert torch.equal(y[:5], x.cpu()[:5]) and (y[5:9] == 0).all() and torch.isnan(y[9])


def put(codes, t):
    """An 8-bit matrix of whole values (codes) times 2^t per row, on the GPU."""
    R, K = codes.shape[-2:]
    s = torch.full((*codes.shape[:-1], W.fp8_scale_cols(K)), 127, dtype=torch.uint8)
    s[..., :-(-K // 128)] = (t + 127).to(torch.uint8)[..., None]
    return W.Fp8Matrix(codes.to(torch.float8_e4m3fn).cuda(), s.cuda().view(torch.float8_e8m0fnu))


@pytest.mark.parametrize("M", [1, 5, 40, 200, 700])
def test_experts_with_gates_at_the_ends(M):
    """Tokens of +-2^120 against gates of 192, 240, 256 and 448: sums of 2.55e38, 3.19e38, and two past 32 bits.  The up
    projection gives +-1, so h is 192 and 240 times 2^120 for the positive tokens and 0 for the negative ones, exactly; down
    brings it back by 2^-120.  A sum past 32 bits counts as the largest value (2^128, 256 here) or as infinite (448)."""
    K, I, N = 32, 16, 16
    gate, up, down = torch.zeros(1, I, K), torch.zeros(1, I, K), torch.zeros(1, N, I)
    gate[0, :4, 0] = torch.tensor([192.0, 240.0, 256.0, 448.0])
    up[0, :4, 0] = 1.0
    down[0, range(N), range(N)] = 1.0
    gu = put(torch.cat([gate, up], 1), torch.cat([torch.zeros(1, I), torch.full((1, I), -120)], 1).long())
    dn = put(down, torch.full((1, N), -120).long())
    x = torch.zeros(M, K, dtype=torch.bfloat16)
    sign = torch.where(torch.arange(M) % 3 == 1, -1.0, 1.0)
    x[:, 0] = sign * 2.0 ** 120
    y = W.w8a8_moe(x.cuda(), torch.zeros(M, 1, dtype=torch.int32, device="cuda"), torch.ones(M, 1, device="cuda"), gu, dn)
    want = torch.zeros(M, N)
    want[sign > 0, :2] = torch.tensor([192.0, 240.0])
    y = y.float().cpu()
    past = y[:, 2:4].clone()
    y[:, 2:4] = 0
    assert torch.equal(y, want)
    assert (past[sign < 0] == 0).all() and (past[sign > 0] >= 256).all() and (past[sign > 0] <= 448).all()
    assert W.awq_last_device_status() == 0
