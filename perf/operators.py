"""Cases of the 8-bit block-scaled operators: the quantizer, the linear layer, the expert router and the expert MLP.

``listed`` and ``draw`` give cases, ``prepare`` makes what a caller has in hand, ``run`` makes one pass -- the plain
torch form, or with ``own`` the library's calls -- and ``exact`` gives the same outputs from the definitions in 64 bits.

An 8-bit matrix is e4m3 codes [rows][K] and one power-of-two scale (e8m0) per row and block of 128 columns, the block
count rounded up to a multiple of 4 (the scales past the last block are 1).  The scale of a block is the smallest power
of two t with max|x| <= 448 t, not below 2^-126; a code is x / t rounded to e4m3, ties to even.
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a projection's weight on its way into the 8-bit format (once per weight, over every weight of a model)
        {"name": "quantize weight", "op": "quantize", "R": 14336, "K": 4096, "type": "fp16"},
        # a ragged batch of activations, the last block of a row only partly filled
        {"name": "quantize ragged", "op": "quantize", "R": 77, "K": 1040, "type": "bf16"},
        # one token of a decode step through a square projection: latency counts
        {"name": "linear decode 1", "op": "linear", "M": 1, "N": 4096, "K": 4096, "type": "fp16"},
        # a decode batch through an up projection: the weight's bytes count
        {"name": "linear decode 16", "op": "linear", "M": 16, "N": 14336, "K": 4096, "type": "bf16"},
        # odd sizes on every side: partial tiles and a partial last block
        {"name": "linear ragged", "op": "linear", "M": 333, "N": 1000, "K": 1040, "type": "fp16"},
        # a prompt through the widest projection: the tensor cores count
        {"name": "linear prompt", "op": "linear", "M": 2048, "N": 28672, "K": 8192, "type": "bf16"},
        # one token's choice among many experts in groups, with a balancing bias
        {"name": "route one token", "op": "route", "M": 1, "E": 256, "topk": 8, "score": "sigmoid", "groups": 8,
         "topk_groups": 4, "bias": True, "renorm": True, "type": "fp32"},
        # the same choice for a long packed prompt
        {"name": "route prompt", "op": "route", "M": 8192, "E": 256, "topk": 8, "score": "sigmoid", "groups": 8,
         "topk_groups": 4, "bias": True, "renorm": True, "type": "fp32"},
        # softmax over an expert count that is no power of two, 16-bit logits with many ties, some experts masked
        {"name": "route softmax", "op": "route", "M": 2047, "E": 60, "topk": 4, "score": "softmax", "groups": 1,
         "topk_groups": 1, "bias": False, "renorm": False, "type": "bf16"},
        # one decode token through two of eight wide experts: the two experts' bytes count
        {"name": "experts decode 1", "op": "moe", "M": 1, "E": 8, "topk": 2, "K": 4096, "I": 14336, "type": "fp16"},
        # odd sizes on every side, some slots of a padded batch without an expert
        {"name": "experts ragged", "op": "moe", "M": 77, "E": 13, "topk": 3, "K": 1040, "I": 656, "type": "bf16"},
        # a prompt through many narrow experts: tensor cores, gather and combine
        {"name": "experts prompt", "op": "moe", "M": 2048, "E": 64, "topk": 6, "K": 4096, "I": 1024, "type": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in lo..hi, even over its logarithm, a multiple of `step`."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, max(step, v // step * step)))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "route", "moe", "moe"])
    while True:
        if op == "quantize":
            c = {"op": op, "R": _log(rng, 1, 65536), "K": _log(rng, 16, 28672, 16), "type": rng.choice(["fp16", "bf16"])}
            small = c["R"] * c["K"] <= 14336 * 8192
        elif op == "linear":
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 8, 28672), "K": _log(rng, 16, 28672, 16),
                 "type": rng.choice(["fp16", "bf16"])}
            small = c["M"] * c["N"] * c["K"] <= 2048 * 28672 * 8192 and c["N"] * c["K"] <= 28672 * 8192
        elif op == "route":
            groups = rng.choice([1, 1, 2, 4, 8])
            per = rng.randint(2, 512 // groups if groups > 1 else 320)
            tg = rng.randint(1, groups)
            c = {"op": op, "M": _log(rng, 1, 16384), "E": groups * per, "topk": rng.randint(1, min(16, tg * per)),
                 "score": rng.choice(["softmax", "sigmoid"]), "groups": groups, "topk_groups": tg,
                 "bias": rng.random() < 0.5, "renorm": rng.random() < 0.5, "type": rng.choice(["fp32", "bf16", "fp16"])}
            small = True
        else:
            E = rng.randint(2, 128)
            c = {"op": op, "M": _log(rng, 1, 4096), "E": E, "topk": rng.randint(1, min(8, E)),
                 "K": _log(rng, 128, 8192, 16), "I": _log(rng, 64, 14336, 16), "type": rng.choice(["fp16", "bf16"])}
            small = E * c["K"] * c["I"] <= 8 * 4096 * 14336 and c["M"] * c["topk"] * c["K"] * c["I"] <= 2048 * 6 * 4096 * 4096
        if small:
            return c


def _blocks(K):
    return (K + BLOCK - 1) // BLOCK


def _matrix_bytes(R, K):
    return R * K + R * _blocks(K)


def work(case):
    c = case
    if c["op"] == "quantize":
        return {"bytes": 2 * c["R"] * c["K"] + _matrix_bytes(c["R"], c["K"]), "flops": 2 * c["R"] * c["K"]}
    if c["op"] == "linear":
        return {"bytes": 2 * c["M"] * c["K"] + _matrix_bytes(c["N"], c["K"]) + 2 * c["M"] * c["N"],
                "flops": 2 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "route":
        return {"bytes": c["M"] * c["E"] * (4 if c["type"] == "fp32" else 2) + 8 * c["M"] * c["topk"],
                "flops": 8 * c["M"] * c["E"]}
    used = c["E"] * (1.0 - (1.0 - c["topk"] / c["E"]) ** c["M"])  # experts that M tokens of random choices reach
    return {"bytes": int(used * (_matrix_bytes(2 * c["I"], c["K"]) + _matrix_bytes(c["K"], c["I"])))
            + 4 * c["M"] * c["K"] + 8 * c["M"] * c["topk"],
            "flops": 6 * c["M"] * c["topk"] * c["K"] * c["I"]}


# ------------------------------------------------------------------------------------------------ inputs
def _activations(g, M, K, dtype):
    x = torch.randn(M, K, device="cuda", generator=g)
    loud = torch.rand(K, device="cuda", generator=g) < 0.01  # about 1 % of the channels are salient
    return (x * torch.where(loud, 20.0, 1.0)).to(dtype)


def _weights(g, R, K):
    """Quantized random weights, made in pieces (codes uint8 [R][K] and scales uint8, as bytes)."""
    codes = torch.empty(R, K, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(R, (_blocks(K) + 3) // 4 * 4, dtype=torch.float8_e8m0fnu, device="cuda")
    step = max(1, (1 << 27) // K)
    for r in range(0, R, step):
        n = min(step, R - r)
        w = torch.randn(n, K, device="cuda", generator=g) * 0.02
        c, s = _quantize(w)
        codes[r:r + n], scales.view(torch.uint8)[r:r + n] = c, s.view(torch.uint8)
    return codes, scales


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[c["type"]]
    s = dict(c)
    if c["op"] == "quantize":
        s["x"] = _activations(g, c["R"], c["K"], dtype)
    elif c["op"] == "linear":
        s["x"] = _activations(g, c["M"], c["K"], dtype)
        s["w"] = _weights(g, c["N"], c["K"])
    elif c["op"] == "route":
        s["logits"] = (torch.randn(c["M"], c["E"], device="cuda", generator=g) * 2.0).to(dtype)
        if c["type"] == "bf16":  # experts that are switched off for some tokens
            s["logits"][torch.rand(c["M"], c["E"], device="cuda", generator=g) < 0.05] = -math.inf
        s["b"] = torch.randn(c["E"], device="cuda", generator=g) * 0.1 if c["bias"] else None
    else:
        s["x"] = _activations(g, c["M"], c["K"], dtype)
        s["ids"] = torch.rand(c["M"], c["E"], device="cuda", generator=g).topk(c["topk"]).indices.to(torch.int32)
        if c["M"] > 8:  # the padded end of a batch has no experts
            s["ids"][c["M"] - c["M"] // 16 - 1:] = -1
        p = torch.rand(c["M"], c["topk"], device="cuda", generator=g) + 0.1
        s["weights"] = p / p.sum(1, keepdim=True)
        cu, su = _weights(g, c["E"] * 2 * c["I"], c["K"])
        cd, sd = _weights(g, c["E"] * c["K"], c["I"])
        s["gate_up"] = cu.view(c["E"], 2 * c["I"], c["K"]), su.view(c["E"], 2 * c["I"], -1)
        s["down"] = cd.view(c["E"], c["K"], c["I"]), sd.view(c["E"], c["K"], -1)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _quantize(x):
    """Codes and scales of x [..., K] (every step exact in 32 bits but the rounding of the codes)."""
    K = x.shape[-1]
    G = _blocks(K)
    v = torch.nn.functional.pad(x.float(), (0, G * BLOCK - K)).unflatten(-1, (G, BLOCK))
    amax = v.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    t = torch.where(amax > 0, e - 9 + (m > 0.875), -126).clamp(min=-126)
    scale = ((t + 127) << 23).view(torch.float32)  # 2^t from its bits
    codes = (v / scale.unsqueeze(-1)).flatten(-2)[..., :K].to(torch.float8_e4m3fn)
    b = torch.nn.functional.pad((t + 127).to(torch.uint8), (0, (G + 3) // 4 * 4 - G), value=127)
    return codes, b.view(torch.float8_e8m0fnu)


def _values(codes, scales):
    """The 32-bit values that codes [..., K] and scales stand for."""
    K = codes.shape[-1]
    t = scales.float()[..., :_blocks(K)].repeat_interleave(BLOCK, dim=-1)[..., :K]
    return codes.float() * t


def _plain_route(s):
    l, E, G = s["logits"].double(), s["E"], s["groups"]
    off = torch.isneginf(l) | torch.isnan(l)
    l = l.clamp(max=torch.finfo(torch.float32).max)
    if s["score"] == "softmax":
        top = l.masked_fill(off, -1e300).amax(1, keepdim=True)
        p = torch.exp(l.masked_fill(off, -1e300) - top).masked_fill(off, 0.0)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = (1.0 / (1.0 + torch.exp(-l))).masked_fill(off, 0.0)
    q = (p if s["b"] is None else p + s["b"].double()).masked_fill(off, -1e300)
    if G > 1:
        of = q.unflatten(1, (G, E // G)).sort(dim=2, descending=True).values[..., :2].sum(2)
        kept = of.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        taken = torch.zeros_like(of, dtype=torch.bool).scatter(1, kept, True)
        q = q.masked_fill(~taken.repeat_interleave(E // G, dim=1), -math.inf)
    ids = q.sort(dim=1, descending=True, stable=True).indices[:, :s["topk"]]
    w = p.gather(1, ids)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.to(torch.int32), (w * 2.5).float()


def _plain_moe(s):
    x, E, I, topk = s["x"], s["E"], s["I"], s["topk"]
    M, K = x.shape
    flat = s["ids"].flatten().long()
    slots = ((flat >= 0) & (flat < E)).nonzero().squeeze(1)
    order = slots[flat[slots].argsort(stable=True)]            # assignments in the order of their experts
    e = flat[order]
    count = torch.bincount(e, minlength=E)
    active = count.nonzero().squeeze(1)
    place = torch.cumsum(count > 0, 0)[e] - 1                   # the expert's place among the active ones
    at = torch.arange(len(e), device=e.device) - (torch.cumsum(count, 0) - count)[e]
    xq = _values(*_quantize(x))
    rows = torch.zeros(len(active), int(count.max()), K, device="cuda")
    rows[place, at] = xq[order // topk]
    pick = lambda m: _values(m[0].view(torch.uint8)[active].view(torch.float8_e4m3fn),  # noqa: E731
                             m[1].view(torch.uint8)[active].view(torch.float8_e8m0fnu))
    ab = torch.bmm(rows, pick(s["gate_up"]).transpose(1, 2))
    a, b = ab[..., :I], ab[..., I:]
    h = _values(*_quantize(a / (1.0 + torch.exp(-a)) * b))
    y = torch.bmm(h, pick(s["down"]).transpose(1, 2))
    out = torch.zeros(M * topk, K, device="cuda")
    out[order] = y[place, at]
    return (out.view(M, topk, K) * s["weights"].unsqueeze(2)).sum(1).to(x.dtype)


def run(state):
    s = state
    if own:
        import weight_only_int4_05_b200 as W

        if s["op"] == "quantize":
            m = W.fp8_quantize(s["x"])
            return m.codes, m.scales
        if s["op"] == "linear":
            return W.w8a8_linear(s["x"], W.Fp8Matrix(*s["w"]))
        if s["op"] == "route":
            r = W.moe_route(s["logits"], s["topk"], score=s["score"], bias=s["b"], groups=s["groups"],
                            topk_groups=s["topk_groups"], renorm=s["renorm"], scale=2.5)
            return r.ids, r.weights
        return W.w8a8_moe(s["x"], s["ids"], s["weights"], W.Fp8Matrix(*s["gate_up"]), W.Fp8Matrix(*s["down"]))
    if s["op"] == "quantize":
        return _quantize(s["x"])
    if s["op"] == "linear":
        return (_values(*_quantize(s["x"])) @ _values(*s["w"]).t()).to(s["x"].dtype)
    if s["op"] == "route":
        return _plain_route(s)
    return _plain_moe(s)


# ------------------------------------------------------------------------------------------------ 64 bits
def _power(t):
    """2^t as a 64-bit float, from its bits (the power function is not exact on every device)."""
    return ((t + 1023) << 52).view(torch.float64)


def _exact_blocks(x):
    """(codes' values, scales per block) of x in 64 bits, by the definition."""
    K = x.shape[-1]
    G = _blocks(K)
    v = torch.cat([x, x.new_zeros(*x.shape[:-1], G * BLOCK - K)], -1).reshape(*x.shape[:-1], G, BLOCK)
    amax = v.abs().amax(-1)
    t = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0)).clamp(min=-126.0).long()
    t = torch.where(amax > 448.0 * _power(t), t + 1, t)            # the logarithm may be off next to a border
    t = torch.where(amax <= 448.0 * _power(t - 1), t - 1, t).clamp(min=-126)
    u = v * _power(-t).unsqueeze(-1)
    low = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))).long()  # e4m3: 3 mantissa bits, least normal 2^-6
    low = torch.where(u.abs() < _power(low), low - 1, low).clamp(min=-6)
    low = torch.where(u.abs() >= _power(low + 1), low + 1, low)
    return (torch.round(u * _power(3 - low)) * _power(low - 3)).reshape(*x.shape[:-1], G * BLOCK)[..., :K], _power(t)


def _exact_grid(x):
    c, t = _exact_blocks(x)
    return c * t.repeat_interleave(BLOCK, -1)[..., :x.shape[-1]]


def _exact_matrix(codes, scales):
    K = codes.shape[-1]
    t = _power(scales.view(torch.uint8).long() - 127)
    return codes.double() * t[..., torch.arange(K, device=codes.device) // BLOCK]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        c, t = _exact_blocks(s["x"].double())
        full = t.new_ones(t.shape[0], (t.shape[1] + 3) // 4 * 4)
        full[:, :t.shape[1]] = t
        return c, full
    if s["op"] == "linear":
        return torch.matmul(_exact_grid(s["x"].double()), _exact_matrix(*s["w"]).T)
    if s["op"] == "route":
        l = s["logits"].double()
        l = torch.where(torch.isnan(l), -math.inf, l)
        off = l == -math.inf
        if s["score"] == "softmax":
            p = torch.softmax(l, 1).nan_to_num(0.0)
        else:
            p = torch.sigmoid(l)
        ids, _ = _plain_route(s)  # whole numbers: compared as they are
        w = torch.where(off, 0.0, p).gather(1, ids.long())
        if s["renorm"]:
            w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
        return None, 2.5 * w
    M, K = s["x"].shape
    xq = _exact_grid(s["x"].double())
    y = xq.new_zeros(M, K)
    for e in range(s["E"]):
        row, slot = (s["ids"] == e).nonzero(as_tuple=True)
        if len(row):
            w = _exact_matrix(s["gate_up"][0][e], s["gate_up"][1][e])
            a, b = (xq[row] @ w.T).chunk(2, 1)
            h = _exact_grid(torch.sigmoid(a) * a * b)
            d = h @ _exact_matrix(s["down"][0][e], s["down"][1][e]).T
            y.index_add_(0, row, d * s["weights"].double()[row, slot].unsqueeze(1))
    return y
