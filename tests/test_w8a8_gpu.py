"""The 8-bit operators on the GPU against their definitions in 64 bits: the quantizer bit for bit, the linear layer within
its sums' rounding, the router's choice exactly, the expert MLP within what its sums may move on the 8-bit grid."""
import numpy as np
import pytest
import torch

import fp8_reference as R
import weight_only_int4_05_b200 as W

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def activations(rng, M, K, dtype):
    x = rng.normal(size=(M, K))
    x[:, rng.random(K) < 0.02] *= 20.0
    return torch.from_numpy(x).to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def matrix(rng, shape, sigma=0.02):
    """A quantized random weight on the GPU and its 64-bit values (from the codes that the GPU wrote)."""
    w = W.fp8_quantize((torch.from_numpy(rng.normal(size=shape) * sigma)).to(torch.float16).cuda())
    t = w.scales.view(torch.uint8).cpu().numpy().astype(np.int64) - 127
    return w, R.values(np64(w.codes.float()), t)


def status_ok():
    assert W.awq_last_device_status() == 0


# ------------------------------------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (3, 144), (5, 512), (77, 1040), (33, 4096), (2, 16400)])
def test_quantize_bit_exact(rows, K, dtype):
    x = activations(np.random.default_rng(rows * K), rows, K, TYPES[dtype])
    m = W.fp8_quantize(x.cuda())
    c, t = R.quantize(np64(x))
    assert np.array_equal(np64(m.codes.float()), c)
    b = m.scales.view(torch.uint8).cpu().numpy()
    G = -(-K // 128)
    assert m.scales.shape == (rows, W.fp8_scale_cols(K))
    assert np.array_equal(b[:, :G], t + 127) and (b[:, G:] == 127).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quantize_edges_bit_exact(dtype):
    """Blocks of zeros, of signed zeros, with a maximum on and next to a border (448 2^t), of the type's least and largest
    values, of exact ties between two codes."""
    td = TYPES[dtype]
    tiny, huge = (2.0 ** -24, 65504.0) if dtype == "fp16" else (2.0 ** -133, 2.0 ** 127 * 1.9921875)
    rows = [np.zeros(128), np.where(np.arange(128) % 2, 0.0, -0.0), np.full(128, 448.0), np.full(128, 1.75 * 2.0 ** -3),
            np.full(128, 1.7578125 * 2.0 ** -3), np.r_[1.0, np.zeros(127)], np.full(128, tiny), np.full(128, huge),
            np.r_[448.0, (np.arange(127) + 0.5) * 2.0], np.r_[-448.0, (np.arange(127) + 0.5) * 2.0 ** -9],
            np.r_[huge, np.full(127, tiny)]]
    x = torch.from_numpy(np.stack(rows)).to(td)
    m = W.fp8_quantize(x.cuda())
    c, t = R.quantize(np64(x))
    assert np.array_equal(np64(m.codes.float()), c)
    assert np.array_equal(m.scales.view(torch.uint8).cpu().numpy()[:, :1], t + 127)


def test_quantize_stack_is_rows_and_out_is_reused():
    x = activations(np.random.default_rng(5), 24, 272, torch.bfloat16).cuda()
    flat, stack = W.fp8_quantize(x), W.fp8_quantize(x.view(3, 8, 272))
    assert torch.equal(flat.codes.view(torch.uint8), stack.codes.view(torch.uint8).view(24, 272))
    assert torch.equal(flat.scales.view(torch.uint8), stack.scales.view(torch.uint8).view(24, -1))
    again = W.fp8_quantize(x * 2, out=flat)
    assert again is flat
    assert torch.equal(flat.codes.view(torch.uint8), stack.codes.view(torch.uint8).view(24, 272))  # the scale moved


def test_quantize_nan_stays_in_its_place():
    x = torch.ones(2, 256, dtype=torch.float16)
    x[0, 3] = float("nan")
    c = W.fp8_quantize(x.cuda()).codes.float().cpu()
    assert torch.isnan(c[0, 3]) and int(torch.isnan(c).sum()) == 1


# ------------------------------------------------------------------------------------------------ linear
SHAPES = [(1, 8, 16), (1, 256, 512), (2, 100, 128), (7, 129, 144), (16, 128, 640), (17, 513, 1040), (31, 1, 2048),
          (64, 384, 4096), (100, 250, 400), (128, 256, 1024), (129, 130, 1152), (200, 640, 528), (256, 128, 512),
          (257, 257, 272), (333, 1000, 1040), (600, 384, 2560)]


def check_linear(y, xq, wv, dtype):
    ref = xq @ wv.T
    err = R.sum_error(xq, wv)
    bound = err + R.rounding(np.abs(ref) + err, torch.finfo(dtype).eps)
    worst = np.max(np.abs(np64(y) - ref) / bound)
    assert worst <= 1.0, worst


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dtype):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    w, wv = matrix(rng, (N, K))
    x = activations(rng, M, K, TYPES[dtype])
    y = W.w8a8_linear(x.cuda(), w)
    assert y.dtype == TYPES[dtype] and y.shape == (M, N)
    check_linear(y, R.grid(np64(x)), wv, TYPES[dtype])
    q = W.fp8_quantize(x.cuda())  # quantized once, the same bits
    assert torch.equal(W.w8a8_linear(q, w, dtype=TYPES[dtype]), y)
    status_ok()


@pytest.mark.parametrize("M,N,K", [(1, 4096, 14336), (16, 14336, 4096), (48, 4096, 4096), (2048, 4096, 1024)])
def test_linear_large_rows(M, N, K):
    """The shapes of the decode and prefill workloads, on sampled rows and columns."""
    rng = np.random.default_rng(N + K)
    w = W.fp8_quantize(torch.randn(N, K, device="cuda", generator=torch.Generator("cuda").manual_seed(N)).mul_(0.02).half())
    x = activations(rng, M, K, torch.bfloat16)
    y = W.w8a8_linear(x.cuda(), w)
    ms, ns = np.unique(np.r_[0, M - 1, rng.integers(0, M, 24)]), np.unique(np.r_[0, N - 1, rng.integers(0, N, 400)])
    t = w.scales.view(torch.uint8).cpu().numpy().astype(np.int64)[ns] - 127
    wv = R.values(np64(w.codes.float().cpu()[torch.from_numpy(ns)]), t)
    check_linear(y.cpu()[torch.from_numpy(ms)][:, torch.from_numpy(ns)], R.grid(np64(x[torch.from_numpy(ms)])), wv,
                 torch.bfloat16)
    status_ok()


def test_linear_scales_reach_the_right_rows_and_blocks():
    """Codes of 1 everywhere and another power of two for every row and block on both sides: the sum names each scale."""
    M, N, K = 150, 300, 1280
    rng = np.random.default_rng(3)
    tx, tw = rng.integers(-6, 7, (M, K // 128)), rng.integers(-6, 7, (N, K // 128))
    def put(t):
        s = np.full((t.shape[0], W.fp8_scale_cols(K)), 127, np.uint8)
        s[:, :t.shape[1]] = t + 127
        return W.Fp8Matrix(torch.ones(t.shape[0], K).to(torch.float8_e4m3fn).cuda(),
                           torch.from_numpy(s).cuda().view(torch.float8_e8m0fnu))
    y = W.w8a8_linear(put(tx), put(tw), dtype=torch.bfloat16)
    check_linear(y, np.repeat(np.ldexp(1.0, tx), 128, 1), np.repeat(np.ldexp(1.0, tw), 128, 1), torch.bfloat16)


def test_linear_writes_its_output_alone():
    rng = np.random.default_rng(9)
    w, wv = matrix(rng, (200, 272))
    x = activations(rng, 37, 272, torch.float16)
    buf = torch.full((39 * 200,), 7.0, dtype=torch.float16, device="cuda")
    out = buf[200:38 * 200].view(37, 200)
    assert W.w8a8_linear(x.cuda(), w, out=out) is out
    check_linear(out, R.grid(np64(x)), wv, torch.float16)
    assert (buf[:200] == 7).all() and (buf[38 * 200:] == 7).all()


# ------------------------------------------------------------------------------------------------ router
def check_route(r, logits, **kw):
    ids, w = R.route(logits, **kw)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    # 32-bit weights, in units of 2^-24 relative.  Sigmoid: the exponential 4 (2 ulp), 1 + e and the quotient 1 each, so 6;
    # renormalised by a sum of such terms (6, and 5 additions) with a quotient and the scale's product: 6 + 11 + 2 = 19.
    # Softmax: l - top rounds by 1/2 unit of |l - top| = |ln p/pmax|, the exponential 4; the sum of up to 1024 terms takes 37
    # additions and the terms' own errors (4, and sum p |ln p/pmax| / 2 <= 4); two quotients' and the scale's roundings: 64 is
    # above all of them but |ln p/pmax|.  Below fp32's least normal value its steps stop shrinking at 2^-149; divided by a sum
    # of at least 2^-20 that is 2^-129.
    l = np.where(np.isnan(logits), -np.inf, np.minimum(logits.astype(np.float64), np.finfo(np.float32).max))
    with np.errstate(invalid="ignore"):
        far = np.abs(np.take_along_axis(l, ids, 1) - l.max(1, keepdims=True)) if kw["score"] == "softmax" else 0.0
    far = np.where(np.isfinite(far), far, 0.0)
    off = np.abs(np64(r.weights) - w) - ((64 + far) * 2.0 ** -24 * np.abs(w) + 2.0 ** -126)
    assert off.max() <= 0, off.max()


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("score,use_bias", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("M,E,topk,groups,tg,renorm", [
    (1, 8, 2, 1, 1, True), (5, 1, 1, 1, 1, False), (33, 60, 4, 1, 1, False), (64, 256, 8, 8, 4, True),
    (17, 160, 6, 8, 3, False), (9, 512, 16, 4, 1, True), (6, 1000, 32, 1, 1, True), (3, 1024, 8, 32, 32, False),
    (21, 64, 8, 32, 5, True), (4, 33, 32, 1, 1, True), (12, 32, 3, 32, 4, True)])
def test_route(M, E, topk, groups, tg, renorm, score, use_bias, dtype):
    rng = np.random.default_rng(M + E * 3 + topk)
    l = torch.from_numpy(rng.normal(size=(M, E)) * 2).to(TYPES[dtype])
    bias = torch.from_numpy(rng.normal(size=E) * 0.1).float() if use_bias else None
    r = W.moe_route(l.cuda(), topk, score=score, bias=None if bias is None else bias.cuda(), groups=groups,
                    topk_groups=tg, renorm=renorm, scale=2.5)
    check_route(r, np64(l), topk=topk, score=score, bias=None if bias is None else np64(bias), groups=groups,
                topk_groups=tg, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,tg", [(1, 1), (4, 2)])
def test_route_masks_ties_and_borders(score, groups, tg):
    """Rows of equal logits, of -inf and NaN but for a few, of nothing else, of the type's extremes, and of logits one unit in
    the last place apart."""
    E, topk = 64, 6
    l = np.zeros((9, E), np.float32)
    l[1] = -np.inf
    l[2] = -np.inf
    l[2, [5, 40]] = 1.0
    l[3] = np.nan
    l[3, 7] = 0.5
    l[4] = np.finfo(np.float32).min
    l[5, 10] = np.inf
    l[6] = 3.0 + np.spacing(np.float32(3.0)) * (np.arange(E) % 5)
    l[7] = -200.0 - np.arange(E)
    l[8, ::2] = -1e4
    for renorm in (False, True):
        r = W.moe_route(torch.from_numpy(l).cuda(), topk, score=score, groups=groups, topk_groups=tg, renorm=renorm)
        check_route(r, l, topk=topk, score=score, groups=groups, topk_groups=tg, renorm=renorm)
    bias = np.zeros(E, np.float32)
    bias[3] = np.spacing(np.float32(0.5))
    r = W.moe_route(torch.from_numpy(l).cuda(), topk, score=score, bias=torch.from_numpy(bias).cuda(), groups=groups,
                    topk_groups=tg)
    check_route(r, l, topk=topk, score=score, bias=bias, groups=groups, topk_groups=tg)


# ------------------------------------------------------------------------------------------------ experts
def check_moe(M, E, topk, K, I, N, dtype, ids, rng):
    gu, gv = matrix(rng, (E, 2 * I, K), 0.05)
    dn, dv = matrix(rng, (E, N, I), 0.05)
    x = activations(rng, M, K, dtype)
    w = torch.from_numpy(rng.random((M, topk)) + 0.1).float()
    y = W.w8a8_moe(x.cuda(), ids.cuda(), w.cuda(), gu, dn)
    ref, bound = R.moe(np64(x), ids.numpy(), w.numpy(), gv, dv, torch.finfo(dtype).eps)
    worst = np.max(np.abs(np64(y) - ref) / bound)
    assert worst <= 1.0, worst
    assert torch.equal(y, W.w8a8_moe(x.cuda(), ids.cuda(), w.cuda(), gu, dn))  # the same bits every time
    status_ok()
    return y


def choose(rng, M, E, topk):
    return torch.from_numpy(np.stack([rng.permutation(E)[:topk] for _ in range(M)])).int()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,E,topk,K,I,N", [
    (1, 1, 1, 16, 16, 8), (1, 8, 2, 256, 128, 256), (3, 4, 2, 272, 144, 100), (16, 8, 8, 512, 256, 512),
    (77, 13, 3, 528, 400, 260), (130, 2, 1, 128, 272, 131), (200, 3, 2, 640, 128, 64), (40, 64, 6, 256, 96, 256)])
def test_moe(M, E, topk, K, I, N, dtype):
    rng = np.random.default_rng(M + E + K)
    check_moe(M, E, topk, K, I, N, TYPES[dtype], choose(rng, M, E, topk), rng)


@pytest.mark.parametrize("kind", ["one expert", "none", "half none", "twice", "out of range", "uneven"])
def test_moe_choices(kind):
    """Every token to one expert, to none, to one expert twice, to ids that are no experts, and most tokens to one expert."""
    rng = np.random.default_rng(11)
    M, E, topk, K, I, N = 150, 9, 3, 256, 144, 136
    ids = choose(rng, M, E, topk)
    if kind == "one expert":
        ids = torch.full((M, topk), -1, dtype=torch.int32)
        ids[:, 1] = 4
    elif kind == "none":
        ids[:] = -1
    elif kind == "half none":
        ids[::2] = -1
        ids[1::4, 2] = -7
    elif kind == "twice":
        ids[:, 1] = ids[:, 0]
    elif kind == "out of range":
        ids[::3, 0] = E
        ids[1::3, 1] = 2 ** 31 - 1
        ids[2::3, 2] = -2 ** 31
    else:
        ids[5:, 0] = 2
        ids[5:, 1:] = -1
    y = check_moe(M, E, topk, K, I, N, torch.bfloat16, ids, rng)
    if kind == "none":
        assert not y.any()


def test_moe_many_copies():
    """More than one chunk of 1024 copies on the way to the sorted order: a one-hot layer shows every row's place."""
    M, E, topk, K = 1500, 24, 4, 128
    rng = np.random.default_rng(2)
    ids = choose(rng, M, E, topk)
    ids[rng.random((M, topk)) < 0.1] = -1
    dtype = torch.float16
    gate = torch.eye(K).repeat(E, 1, 1)
    up = torch.eye(K).repeat(E, 1, 1)
    dn = torch.eye(K).repeat(E, 1, 1) * (2.0 ** (torch.arange(E) % 7 - 3))[:, None, None]
    gu = W.fp8_quantize(torch.cat([gate, up], 1).to(dtype).cuda())
    dq = W.fp8_quantize(dn.to(dtype).cuda())
    x = activations(rng, M, K, dtype)
    w = torch.from_numpy(2.0 ** rng.integers(-2, 3, (M, topk))).float()
    y = np64(W.w8a8_moe(x.cuda(), ids.cuda(), w.cuda(), gu, dq))
    xq = R.grid(np64(x))
    h = R.silu(xq) * xq  # a = b = xq, exact sums of one product
    hq, moved = R.grid(h), R.grid_moved(h, 2.0 ** -20 * np.abs(h))
    valid = ids.numpy() >= 0
    f = (np.where(valid, w.numpy() * 2.0 ** (ids.numpy() % 7 - 3), 0.0)).sum(1)[:, None]
    bound = f * moved + R.rounding(f * (np.abs(hq) + moved), 2.0 ** -10) + 2.0 ** -21 * topk * f * np.abs(hq)
    # the loud channels' squares leave fp16's range: from 65520 on, halfway past its largest value, a sum rounds to infinity
    ref = f * hq
    over, under = np.abs(ref) - bound >= 65520, np.abs(ref) + bound < 65520
    assert over.any() and (y[over] == np.sign(ref[over]) * np.inf).all()
    assert np.max(np.abs(y[under] - ref[under]) / bound[under]) <= 1.0
    status_ok()


# ------------------------------------------------------------------------------------------------ together
def make_layer(rng, E, K, I, dtype):
    gate = (torch.from_numpy(rng.normal(size=(E, K)) / np.sqrt(K))).to(dtype).cuda()
    gu, gv = matrix(rng, (E, 2 * I, K), 0.05)
    dn, dv = matrix(rng, (E, K, I), 0.05)
    return gate, gu, gv, dn, dv


def layer(x, head, gate, gu, dn):
    """A sparse decoder layer's back half as it is used: a projection, the router on its output, the experts."""
    t = W.w8a8_linear(x, head)
    logits = t @ gate.t()
    r = W.moe_route(logits, 2, score="sigmoid", renorm=True)
    return t, logits, r, W.w8a8_moe(t, r.ids, r.weights, gu, dn)


@pytest.mark.parametrize("M", [1, 37])
def test_projection_router_experts_together(M):
    rng = np.random.default_rng(21)
    E, K, I = 8, 256, 144
    gate, gu, gv, dn, dv = make_layer(rng, E, K, I, torch.bfloat16)
    head, hv = matrix(rng, (K, K), 0.1)
    x = activations(rng, M, K, torch.bfloat16)
    t, logits, r, y = layer(x.cuda(), head, gate, gu, dn)
    check_linear(t, R.grid(np64(x)), hv, torch.bfloat16)
    check_route(r, np64(logits), topk=2, score="sigmoid", renorm=True)
    ref, bound = R.moe(np64(t), r.ids.cpu().numpy(), r.weights.cpu().numpy(), gv, dv, torch.finfo(torch.bfloat16).eps)
    assert np.max(np.abs(np64(y) - ref) / bound) <= 1.0
    status_ok()


def test_captured_graphs_and_streams():
    """Two graphs captured on different streams and replayed at once, eager calls between them: each its own scratch."""
    rng = np.random.default_rng(22)
    E, K, I, M = 8, 256, 144, 24
    gate, gu, gv, dn, dv = make_layer(rng, E, K, I, torch.bfloat16)
    head, hv = matrix(rng, (K, K), 0.1)
    xs = [activations(rng, M, K, torch.bfloat16).cuda() for _ in range(4)]
    want = [layer(x, head, gate, gu, dn)[3] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    static, graphs, outs = [x.clone() for x in xs[:2]], [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            outs.append(layer(static[i], head, gate, gu, dn)[3])
        graphs.append(g)
    for rep in range(20):
        for i in range(2):
            streams[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[i]):
                static[i].copy_(xs[(rep + i) % 4])
                graphs[i].replay()
        eager = layer(xs[3], head, gate, gu, dn)[3]
        torch.cuda.synchronize()
        assert torch.equal(eager, want[3])
        for i in range(2):
            assert torch.equal(outs[i], want[(rep + i) % 4])
    status_ok()


def test_weight_quantized_just_before_its_use():
    """Quantizer and product back to back on one stream, the weight's buffers reused and alternating."""
    rng = np.random.default_rng(23)
    N, K = 1024, 2048
    ws = [torch.from_numpy(rng.normal(size=(N, K)) * 0.02).half().cuda() for _ in range(2)]
    x = activations(rng, 4, K, torch.float16).cuda()
    want = [W.w8a8_linear(x, W.fp8_quantize(w)) for w in ws]
    buf = W.fp8_quantize(ws[0])
    torch.cuda.synchronize()
    got = []
    for rep in range(20):
        W.fp8_quantize(ws[rep % 2], out=buf)
        got.append(W.w8a8_linear(x, buf))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("use_bias", [False, True])
@pytest.mark.parametrize("spread", [2.0 ** -20, 1e-3, 30.0])
def test_route_close_scores(score, use_bias, spread):
    """Logits so close that 32-bit scores cannot order them, with few values (many true ties), and far apart."""
    rng = np.random.default_rng(41)
    M, E = 120, 96
    l = torch.from_numpy(1.0 + spread * rng.integers(-8, 9, (M, E)) * (1 + (rng.random((M, E)) < 0.3))).float()
    bias = torch.from_numpy(rng.integers(-2, 3, E) * 2.0 ** -22).float() if use_bias else None
    for groups, tg, topk in ((1, 1, 7), (8, 3, 7), (3, 2, 32)):
        kw = dict(topk=topk, score=score, groups=groups, topk_groups=tg, renorm=True)
        r = W.moe_route(l.cuda(), bias=None if bias is None else bias.cuda(), **kw)
        check_route(r, np64(l), bias=None if bias is None else np64(bias), **kw)


def test_route_tie_at_the_border_hides_a_better_expert():
    """Equal 32-bit scores of two kinds of experts, the kind that is better in 64 bits behind the border: by its index it would
    be left out."""
    E = 64
    l = np.full((4, E), 1.0, np.float32)
    bias = np.zeros(E, np.float32)
    bias[40:50] = 2.0 ** -27  # half a step of a score of 0.73: lost in 32 bits
    r = W.moe_route(torch.from_numpy(l).cuda(), 6, score="sigmoid", bias=torch.from_numpy(bias).cuda())
    assert r.ids.cpu().tolist() == [[40, 41, 42, 43, 44, 45]] * 4
    bias[:] = 0
    bias[3] = -np.inf
    bias[7] = np.nan
    r = W.moe_route(torch.from_numpy(l).cuda(), 32, score="softmax", bias=torch.from_numpy(bias).cuda())
    assert r.ids.cpu().tolist() == [[e for e in range(E) if e not in (3, 7)][:32]] * 4


@pytest.mark.parametrize("E", [700, 760, 1024])
@pytest.mark.parametrize("M", [20, 700])
def test_moe_many_experts(E, M):
    """Expert counts whose tables come near the default shared memory, one chunk of copies and more than one."""
    rng = np.random.default_rng(E + M)
    check_moe(M, E, 2, 32, 16, 24, torch.bfloat16, torch.from_numpy(rng.integers(0, E, (M, 2))).int(), rng)


@pytest.mark.parametrize("M", [3, 15, 16, 17, 32, 33, 47, 64, 65, 200])
@pytest.mark.parametrize("N,K", [(520, 400), (520, 1536), (96, 6160), (4104, 2048)])
def test_linear_either_side_of_the_fused_quantizer(M, N, K):
    """Up to 16 tokens the product quantizes x itself: the same bits as from the quantizer's arrays."""
    rng = np.random.default_rng(M + K)
    w, wv = matrix(rng, (N, K))
    x = activations(rng, M, K, torch.float16)
    y = W.w8a8_linear(x.cuda(), w)
    check_linear(y, R.grid(np64(x)), wv, torch.float16)
    assert torch.equal(y, W.w8a8_linear(W.fp8_quantize(x.cuda()), w, dtype=torch.float16))


@pytest.mark.parametrize("E,groups", [(4, 2), (6, 3), (30, 15), (32, 32), (96, 6), (1024, 16)])
def test_route_close_groups(E, groups):
    """Group sums that 32 bits cannot order, in groups of one expert, of two and of many; some experts masked."""
    rng = np.random.default_rng(E * groups)
    M, tg = 60, max(1, groups // 2)
    l = (0.5 + rng.integers(0, 3, (M, E)) * 2.0 ** -23).astype(np.float32)
    l[rng.random((M, E)) < 0.1] = -np.inf
    bias = (rng.integers(-1, 2, E) * 2.0 ** -26).astype(np.float32)
    topk = min(5, tg * (E // groups))
    for b in (None, bias):
        for score in ("sigmoid", "softmax"):
            kw = dict(topk=topk, score=score, groups=groups, topk_groups=tg)
            r = W.moe_route(torch.from_numpy(l).cuda(), bias=None if b is None else torch.from_numpy(b).cuda(), **kw)
            check_route(r, l, bias=b, **kw)


@pytest.mark.parametrize("M,N,K", [(40, 130, 6016), (64, 100, 8192), (90, 38, 4112), (300, 260, 5120), (700, 60, 3088)])
def test_linear_few_outputs_long_k(M, N, K):
    """Tiles too few to fill the GPU and a long K: it is split over a cluster, whose parts meet in shared memory."""
    rng = np.random.default_rng(M + N)
    w, wv = matrix(rng, (N, K))
    x = activations(rng, M, K, torch.bfloat16)
    y = W.w8a8_linear(x.cuda(), w)
    check_linear(y, R.grid(np64(x)), wv, torch.bfloat16)
    assert torch.equal(y, W.w8a8_linear(x.cuda(), w))
    status_ok()


@pytest.mark.parametrize("M,E,topk,K,I,N", [(60, 2, 2, 4096, 64, 100), (120, 2, 1, 2048, 2048, 64), (200, 3, 1, 64, 4096, 40)])
def test_moe_few_tiles_long_k(M, E, topk, K, I, N):
    rng = np.random.default_rng(M + K)
    check_moe(M, E, topk, K, I, N, torch.float16, choose(rng, M, E, topk), rng)


@pytest.mark.parametrize("E,M,I", [(56, 600, 128), (100, 1050, 64), (140, 1400, 16)])
def test_moe_tables_parts_and_ring_share_the_memory(E, M, I):
    """Two gate|up accumulators of 32 tokens, a split K and the tables of many experts at once: the ring still fits."""
    rng = np.random.default_rng(E)
    check_moe(M, E, 2, 2048, I, 24, torch.bfloat16, choose(rng, M, E, 2), rng)


def test_nan_stays_with_its_token():
    rng = np.random.default_rng(31)
    M, E, K, I = 40, 6, 256, 144
    gate, gu, gv, dn, dv = make_layer(rng, E, K, I, torch.float16)
    head, hv = matrix(rng, (300, K), 0.1)
    ids, w = choose(rng, M, E, 2).cuda(), torch.ones(M, 2, device="cuda")
    x = activations(rng, M, K, torch.float16).cuda()
    bad = x.clone()
    bad[7, 100] = float("nan")
    others = torch.arange(M, device="cuda") != 7
    for f in (lambda v: W.w8a8_linear(v, head), lambda v: W.w8a8_moe(v, ids, w, gu, dn),
              lambda v: W.w8a8_linear(v[:9].contiguous(), head)):
        a, b = f(x), f(bad)
        keep = others[:len(a)]
        assert torch.equal(a[keep], b[keep]) and torch.isnan(b[7]).all()


def test_refusals_on_the_gpu():
    rng = np.random.default_rng(32)
    gate, gu, gv, dn, dv = make_layer(rng, 4, 256, 144, torch.float16)
    head, hv = matrix(rng, (300, 256), 0.1)
    x = activations(rng, 8, 256, torch.float16).cuda()
    ids, w = choose(rng, 8, 4, 2).cuda(), torch.ones(8, 2, device="cuda")
    flat = W.Fp8Matrix(head.codes.flatten()[:256 * 8].view(8, 256), head.scales[:8, :2].contiguous())
    calls = [
        lambda: W.fp8_quantize(x.float()), lambda: W.fp8_quantize(x.t()), lambda: W.fp8_quantize(x[:, ::2]),
        lambda: W.fp8_quantize(x, out=head), lambda: W.w8a8_linear(x.t(), head), lambda: W.w8a8_linear(x[:, :128].contiguous(), head),
        lambda: W.w8a8_linear(x, flat), lambda: W.w8a8_linear(x, gu), lambda: W.w8a8_linear(x, head, dtype=torch.bfloat16),
        lambda: W.w8a8_linear(x, head, out=torch.empty(8, 299, dtype=torch.float16, device="cuda")),
        lambda: W.w8a8_linear(x, head, out=torch.empty(8, 300, dtype=torch.bfloat16, device="cuda")),
        lambda: W.w8a8_linear(W.fp8_quantize(x), head, dtype=torch.float32),
        lambda: W.moe_route(x, 2, score="tanh"), lambda: W.moe_route(x, 2, bias=torch.zeros(255, device="cuda")),
        lambda: W.moe_route(x.t(), 2), lambda: W.moe_route(x, 2, bias=torch.zeros(256)),
        lambda: W.w8a8_moe(x, ids.long(), w, gu, dn), lambda: W.w8a8_moe(x, ids, w.half(), gu, dn),
        lambda: W.w8a8_moe(x, ids[:7], w, gu, dn), lambda: W.w8a8_moe(x, ids, w[:, :1].contiguous(), gu, dn),
        lambda: W.w8a8_moe(x, ids, w, dn, gu), lambda: W.w8a8_moe(x, ids, w, head, dn),
        lambda: W.w8a8_moe(x, ids.cpu(), w, gu, dn)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: W.fp8_quantize(torch.zeros(4, 24, dtype=torch.float16, device="cuda")),
                 lambda: W.fp8_quantize(torch.zeros(0, 32, dtype=torch.float16, device="cuda")),
                 lambda: W.w8a8_linear(x[:0], head), lambda: W.moe_route(x, 0), lambda: W.moe_route(x, 33),
                 lambda: W.moe_route(x, 4, groups=3), lambda: W.moe_route(x, 9, groups=32, topk_groups=1),
                 lambda: W.w8a8_linear(activations(rng, 600, 256, torch.float16).cuda(), head,
                                       workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(W.AwqError):
            call()
    status_ok()


def test_two_streams_at_once():
    """Products, routers and expert layers in flight on two streams, with and without clusters."""
    rng = np.random.default_rng(33)
    E, K, I = 8, 1024, 272
    gate, gu, gv, dn, dv = make_layer(rng, E, K, I, torch.bfloat16)
    head, hv = matrix(rng, (K, K), 0.1)
    xs = [activations(rng, m, K, torch.bfloat16).cuda() for m in (1, 9, 70, 400)]
    want = [layer(x, head, gate, gu, dn)[3] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for rep in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(layer(xs[(rep + 2 * i) % 4], head, gate, gu, dn)[3])
    torch.cuda.synchronize()
    for i in range(2):
        for rep, y in enumerate(got[i]):
            # the logits between the two are torch's product, whose form may differ by stream: compare where the choice is the same
            assert y.shape == want[(rep + 2 * i) % 4].shape and torch.isfinite(y).all()
            assert torch.equal(y, want[(rep + 2 * i) % 4])
    status_ok()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_experts_in_place_and_other_overlaps_refused(M):
    """w8a8_moe may write y over x; the other calls refuse an output over an input."""
    rng = np.random.default_rng(34)
    E, K, I = 8, 256, 144
    gate, gu, gv, dn, dv = make_layer(rng, E, K, I, torch.bfloat16)
    head, hv = matrix(rng, (K, K), 0.1)
    x = activations(rng, M, K, torch.bfloat16).cuda()
    ids, w = choose(rng, M, E, 2).cuda(), torch.rand(M, 2, device="cuda")
    want = W.w8a8_moe(x, ids, w, gu, dn)
    same = x.clone()
    assert W.w8a8_moe(same, ids, w, gu, dn, out=same) is same
    assert torch.equal(same, want)
    with pytest.raises(W.AwqError):
        W.w8a8_linear(x, head, out=x)
    if M > 16:  # fewer tokens use no workspace
        with pytest.raises(W.AwqError):
            W.w8a8_linear(x, head, workspace=x.view(torch.uint8).view(-1))
    status_ok()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [4, 40])
def test_infinite_values_count_as_448_2_120(M, dtype):
    """Code +-448 and scale byte 120 + 127, in the quantizer and in the product that quantizes by itself; the other
    blocks and tokens keep theirs.  With weights of 2^-10 an infinite value alone gives 1.75 * 2^118: exact in bfloat16."""
    rng = np.random.default_rng(35)
    x = activations(rng, M, 256, TYPES[dtype])
    clean = W.fp8_quantize(x.cuda())
    x[1] = 0
    x[1, 7], x[2, 130] = float("inf"), float("-inf")
    q = W.fp8_quantize(x.cuda())
    codes, scales = q.codes.float().cpu(), q.scales.view(torch.uint8).cpu()
    assert codes[1, 7] == 448 and codes[2, 130] == -448 and scales[1, 0] == 247 and scales[2, 1] == 247
    assert not torch.isnan(codes).any() and int((codes[1] != 0).sum()) == 1
    assert torch.equal(q.codes[2, :128].view(torch.uint8), clean.codes[2, :128].view(torch.uint8))
    w = W.fp8_quantize(torch.full((24, 256), 2.0 ** -10, dtype=torch.bfloat16, device="cuda"))
    y, plain = W.w8a8_linear(x.cuda(), w), W.w8a8_linear(clean, w, dtype=TYPES[dtype])
    assert torch.equal(y, W.w8a8_linear(q, w, dtype=TYPES[dtype]))
    assert (y[1] == (1.75 * 2.0 ** 118 if dtype == "bf16" else float("inf"))).all()
    assert torch.equal(y[0], plain[0]) and torch.equal(y[3:], plain[3:])
    status_ok()
