"""The router's weights within the 32-bit roundings that their computation makes, counted one by one."""
import numpy as np
import pytest
import torch

import fp8_reference as R
import weight_only_int4_05_b200 as W

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def units(l, ids, score, renorm):
    """Relative error of a weight in units of 2^-24 (half a step of a 32-bit value).

    Sigmoid: the exponential is off by 2 units in the last place, 4; 1 + e and the quotient 1 each: 6.  With renorm the sum of up to
    32 such scores has 6 and 5 additions, and there is one more quotient: 6 + 11 + 1.  Softmax: l - top is off by 1/2 unit in the
    last place, which moves the exponential by |l - top| of these units, and 4 more.  Without renorm it is divided (1) by the sum
    of E: each term's own error, weighted by the terms, 31 / 32 E additions in a lane and 5 between lanes; with renorm by the
    chosen ones' sum: at most the worst of the chosen, and 5.  The product with scale: 1."""
    if score == "sigmoid":
        return 6.0 + (12.0 if renorm else 0.0) + 1.0
    far = l.max(1, keepdims=True) - l
    own = np.take_along_axis(far, ids, 1) + 4.0
    if renorm:
        return own + own.max(1, keepdims=True) + 5.0 + 2.0
    p = np.exp(-far)
    mean = (p * far).sum(1, keepdims=True) / p.sum(1, keepdims=True)
    return own + mean + 4.0 + (-(-l.shape[1] // 32) - 1) + 5.0 + 2.0


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("M,E,topk,groups,tg", [(700, 8, 2, 1, 1), (700, 60, 4, 1, 1), (700, 256, 8, 8, 4), (150, 1024, 32, 1, 1)])
def test_weights(M, E, topk, groups, tg, renorm, score, dtype):
    rng = np.random.default_rng(E + topk)
    t = torch.from_numpy(rng.normal(size=(M, E)) * 3).to(TYPES[dtype])
    l = t.double().numpy()
    kw = dict(topk=topk, score=score, groups=groups, topk_groups=tg, renorm=renorm, scale=2.5)
    r = W.moe_route(t.cuda(), **kw)
    ids, w = R.route(l, **kw)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    off = np.abs(r.weights.double().cpu().numpy() - w) / (np.abs(w) * 2.0 ** -24)
    assert (off <= units(l, ids, score, renorm)).all(), (off - units(l, ids, score, renorm)).max()
