"""The router's order where experts' (or groups') 32-bit errors are unlike: a large score that its bias cancels beside small
scores.  The choice has to be that of the 64-bit values in every row."""
import numpy as np
import pytest
import torch

import fp8_reference as R
import route_inputs
import weight_only_int4_05_b200 as W

pytestmark = pytest.mark.gpu


def ids_of(l, bias, **kw):
    r = W.moe_route(torch.from_numpy(l).cuda(), bias=torch.from_numpy(bias).cuda(), **kw)
    return r.ids.cpu().numpy(), R.route(l, bias=bias, **kw)[0]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,topk", [(16, 1), (64, 6), (256, 8), (500, 3)])
def test_a_large_score_cancelled_by_its_bias(E, topk, score):
    l, bias = route_inputs.cancelled_scores(1500, E, topk, score, E)
    got, want = ids_of(l, bias, topk=topk, score=score)
    assert np.array_equal(got, want), f"{(got != want).any(1).sum()} of {len(l)} rows"


def test_two_rows_worked_out_by_hand():
    """The last expert wins in 64 bits (0.00100001424 over 0.00100000934) and, in the second row, the first (2.5e-8 over 2.0e-8);
    in 32 bits the biased one comes last of the three."""
    for l, bias, want in (([-6.9067454, -6.9067554, 1.1229205], [0, 0, -0.75353], 2),
                          ([0.10005, -17.73, -18.4, -60], [-0.52499163, 0, 0, 0], 0)):
        got, ref = ids_of(np.array([l], np.float32), np.array(bias, np.float32), topk=1, score="sigmoid")
        assert ref.tolist() == [[want]] and got.tolist() == [[want]]
