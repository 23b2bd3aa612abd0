"""The scored router's choice where float keys cannot tell the experts or the
groups apart: the 64-bit rule decides, whatever other groups hold, and scores
that a sigmoid or a softmax has rounded to one value still follow their logits."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_b200 as moe
from tests import routed_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [12, 16])  # groups that are not whole lanes, and groups that are
@pytest.mark.parametrize("left", [0, 1])    # experts of the masked group that are not masked
def test_masked_group_beside_large_opposite_biases(size, left):
    # the other groups' two largest keys are s + 64 and s' - 64, their sums a few 1e-6 apart
    T, G = 64, 8
    g = torch.Generator().manual_seed(14)
    bias = torch.full((G, size), -1000.0)
    bias[:, 3], bias[:, 9] = 64.0, -64.0
    bias[5, left:] = -float("inf")
    bias = bias.reshape(-1).cuda()
    l = (torch.randn(T, G * size, generator=g) * 1e-5).cuda()
    ids, w = moe.route_scored(l, 2, bias=bias, n_groups=G, topk_groups=3, group_score="top2")
    r_ids, r_w, tol = ref.route(l.double().cpu().numpy(), 2, bias.double().cpu().numpy(), "sigmoid", G, 3, "top2", True,
                                1.0)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    assert (np.abs(w.double().cpu().numpy() - r_w) <= tol).all()
