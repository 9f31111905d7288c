"""The router's groups where their sums' 32-bit errors are unlike: two biases of +-1000 that cancel in one group."""
import numpy as np
import pytest
import torch

import fp8_reference as R
import route_inputs
import weight_only_int4_05_b200 as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,per,tg", [(8, 2, 3), (8, 8, 4), (16, 4, 5), (32, 4, 8)])
def test_groups_whose_biases_cancel(groups, per, tg):
    l, bias = route_inputs.cancelled_groups(1500, groups, per, groups + per)
    kw = dict(topk=2 * tg, score="sigmoid", groups=groups, topk_groups=tg)
    r = W.moe_route(torch.from_numpy(l).cuda(), bias=torch.from_numpy(bias).cuda(), **kw)
    got, want = r.ids.cpu().numpy(), R.route(l, bias=bias, **kw)[0]
    assert np.array_equal(got, want), f"{(got != want).any(1).sum()} of {len(l)} rows"
