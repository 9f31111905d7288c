"""The 8-bit operators from their definitions in 64 bits (numpy), and how far a kernel's 32-bit sums may move them.

Grid: per row and block of 128 columns, t the smallest whole number >= -126 with max|x| <= 448 2^t; codes are x 2^-t
rounded to e4m3 (3 mantissa bits, least normal 2^-6, so steps of 2^-9 below it), ties to even."""
import numpy as np

BLOCK = 128


def pad_blocks(x):
    K = x.shape[-1]
    G = -(-K // BLOCK)
    v = np.zeros(x.shape[:-1] + (G * BLOCK,))
    v[..., :K] = x
    return v.reshape(x.shape[:-1] + (G, BLOCK))


def exponents(amax):
    """The smallest t >= -126 with amax <= 448 2^t."""
    m, e = np.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1, and 448 = 0.875 2^9
    return np.maximum(np.where(amax > 0, e - 9 + (m > 0.875), -126), -126).astype(np.int64)


def e4m3(u):
    """Nearest e4m3 value, ties to even, of |u| <= 448."""
    _, e = np.frexp(u)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(u / step) * step


def quantize(x):
    """(codes' values [..., K], exponents [..., G]) of x in 64 bits."""
    v = pad_blocks(np.asarray(x, np.float64))
    t = exponents(np.abs(v).max(-1))
    c = e4m3(np.ldexp(v, -t[..., None]))
    return c.reshape(x.shape[:-1] + (-1,))[..., :x.shape[-1]], t


def values(codes, t):
    K = codes.shape[-1]
    return codes * np.ldexp(1.0, np.repeat(t, BLOCK, axis=-1)[..., :K])


def grid(x):
    return values(*quantize(x))


def silu(a):
    return a / (1.0 + np.exp(-a))


def sum_error(x, w):
    """Bound on the error of a 32-bit sum of the exact products x . w, [M][N].  The tensor cores take 32 products at a time
    and add them to the accumulator; each such step keeps at least 22 bits below the largest magnitude involved, and no
    magnitude exceeds S = sum |x||w|: (K / 32 + 1) steps of 2^-22 S."""
    S = np.abs(x) @ np.abs(w).T
    return (x.shape[-1] / 32 + 1) * 2.0 ** -22 * S


def rounding(y, eps):
    """Half a step of the output type (eps = finfo.eps) at |y|, with the least normal range of fp16 added."""
    return np.abs(y) * eps / 2 + 2.0 ** -25


def grid_moved(h, e):
    """How far the grid's values may move, [...][I], when h is off by at most e: the code's two ends, and where the block's
    scale itself may flip, half a step of the coarser scale's smallest steps more."""
    v, d = pad_blocks(h), pad_blocks(e)
    lo_amax = np.maximum(np.abs(v) - d, 0).max(-1)
    t0, t1 = exponents(lo_amax), exponents((np.abs(v) + d).max(-1))
    t = np.where(t1 > t0, t1, t0)[..., None]
    ends = [np.ldexp(e4m3(np.clip(np.ldexp(v + s * d, -t), -448, 448)), t) for s in (-1, 1)]
    moved = ends[1] - ends[0] + np.where((t1 > t0)[..., None], np.ldexp(2.0 ** -9, t), 0.0)
    return moved.reshape(h.shape[:-1] + (-1,))[..., :h.shape[-1]]


def route(logits, topk, score, bias=None, groups=1, topk_groups=1, renorm=False, scale=1.0):
    """ids and weights, token by token, in 64 bits."""
    M, E = logits.shape
    ids, weights = np.zeros((M, topk), np.int64), np.zeros((M, topk))
    for m in range(M):
        l = np.minimum(logits[m].astype(np.float64), np.finfo(np.float32).max)
        off = np.isnan(l) | (l == -np.inf)
        l = np.where(off, -np.inf, l)
        if off.all():
            p = np.zeros(E)
        elif score == "softmax":
            p = np.exp(l - l[~off].max())
            p /= p.sum()
        else:
            with np.errstate(over="ignore"):
                p = 1.0 / (1.0 + np.exp(-l))
        q = p if bias is None else p + bias.astype(np.float64)
        q = np.where(off, -1e300, q)
        order = []
        per = E // groups
        if groups > 1:
            of = [np.sort(q[g * per:(g + 1) * per])[::-1][:2].sum() for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-of[g], g))[:topk_groups]
        else:
            kept = [0]
        order = sorted((e for g in kept for e in range(g * per, (g + 1) * per)), key=lambda e: (-q[e], e))[:topk]
        w = p[order]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(topk)
        ids[m], weights[m] = order, w * scale
    return ids, weights


def moe(x, ids, weights, gate_up, down, eps):
    """(y [M][N], bound on a kernel's error) of the expert MLP; gate_up [E][2 I][K] and down [E][N][I] as 64-bit values."""
    M, I = x.shape[0], down.shape[2]
    xq = grid(x)
    y, err = np.zeros((M, down.shape[1])), np.zeros((M, down.shape[1]))
    for m in range(M):
        for j in range(ids.shape[1]):
            e = ids[m, j]
            if not 0 <= e < len(gate_up):
                continue
            a, b = (xq[m] @ gate_up[e].T).reshape(2, I)
            ea, eb = sum_error(xq[m:m + 1], gate_up[e]).reshape(2, I)
            # |silu'| <= 1.1; the fp32 silu and product add a few units of 2^-24: 2^-20 covers expf, the division and both roundings
            eh = 1.1 * np.abs(b) * ea + np.abs(silu(a)) * eb + 1.1 * ea * eb + 2.0 ** -20 * np.abs(silu(a) * b)
            h = silu(a) * b
            hq = grid(h)
            moved = grid_moved(h, eh)
            d = hq @ down[e].T
            ed = moved @ np.abs(down[e]).T + sum_error((np.abs(hq) + moved)[None], down[e])[0]
            w = float(weights[m, j])
            y[m] += w * d
            err[m] += abs(w) * (ed + 2.0 ** -22 * ids.shape[1] * np.abs(d))
    return y, err + rounding(np.abs(y) + err, eps)
