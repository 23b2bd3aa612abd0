"""The scored router's choice where float keys cannot tell the experts or the
groups apart: the 64-bit rule decides, whatever other groups hold, and scores
that a sigmoid or a softmax has rounded to one value still follow their logits."""
from fractions import Fraction

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


# A score as one of 0, 1/2, 1 plus a 64-bit rest, so that scores next to these stay apart.
def _sigmoid(l):
    if l > 1:
        return Fraction(1) - Fraction(float(np.exp(-l) / (1 + np.exp(-l))))
    if l >= -1:
        return Fraction(1, 2) + Fraction(float(0.5 * np.tanh(0.5 * l)))
    return Fraction(float(np.exp(l) / (1 + np.exp(l))))


def _choice(l, k, bias, n_groups=1, topk_groups=1, group_top=1):
    E = len(l)
    m = E // n_groups
    key = [_sigmoid(float(l[e])) + Fraction(float(bias[e])) for e in range(E)]
    score = [sum(sorted(key[g * m:(g + 1) * m])[-group_top:]) for g in range(n_groups)]
    open_ = sorted(range(n_groups), key=lambda g: (-score[g], g))[:topk_groups]
    return sorted((e for e in range(E) if e // m in open_), key=lambda e: (-key[e], e))[:k]


def _saturated(T, E, seed):
    # above 37 a sigmoid's 64-bit value is 1
    return 38 + 60 * torch.rand(T, E, generator=torch.Generator().manual_seed(seed))


# up to 32 close keys, more than 32, and more than 32 experts chosen
@pytest.mark.parametrize("E,k", [(20, 6), (64, 8), (100, 40), (600, 8)])
def test_saturated_scores_follow_their_logits(E, k):
    l = _saturated(9, E, E)
    l[1] = l[1].half().float() // 1  # equal logits among them: the lower index
    l[2, ::2] -= 80  # half of them far from saturated
    l = l.cuda()
    want, _ = moe.route_scored(l, k)
    got, _ = moe.route_scored(l, k, bias=torch.zeros(E).cuda())
    assert torch.equal(want, got)
    b = torch.randint(0, 3, (E,), generator=torch.Generator().manual_seed(E)).float() * 2.0 ** -24 + 0.25
    got, _ = moe.route_scored(l, k, bias=b.cuda())
    for t, row in enumerate(got.tolist()):
        assert row == _choice(l[t].cpu().numpy(), k, b.numpy())


@pytest.mark.parametrize("size", [8, 12])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_of_saturated_scores(size, group_top, biased):
    G, k = 8, 6
    E = G * size
    l = _saturated(24, E, size + group_top)
    b = torch.randint(0, 2, (E,), generator=torch.Generator().manual_seed(2)).float() * 2.0 ** -24 - 0.5
    ids, _ = moe.route_scored(l.cuda(), k, bias=b.cuda() if biased else None, n_groups=G, topk_groups=3,
                              group_score=group_top)
    for t, row in enumerate(ids.tolist()):
        assert row == _choice(l[t].numpy(), k, b.numpy() if biased else np.zeros(E), G, 3, group_top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("std", [1e-20, 1e-12])
def test_scores_next_to_uniform_follow_their_logits(score, std):
    for E, k in ((24, 6), (96, 40)):
        l = (torch.randn(7, E, generator=torch.Generator().manual_seed(E)) * std).cuda()
        want, _ = moe.route_scored(l, k, score=score)
        got, _ = moe.route_scored(l, k, score=score, bias=torch.full((E,), 0.125).cuda())
        assert torch.equal(want, got)


def test_all_keys_equal():
    for bias in (0.0, -0.5, 1e30, -float("inf")):
        for value in (0.0, 90.0, -200.0):
            l = torch.full((3, 256), value).cuda()
            ids, _ = moe.route_scored(l, 40, bias=torch.full((256,), bias).cuda(), n_groups=8, topk_groups=4,
                                      group_score="top2")
            assert (ids == torch.arange(40).cuda()).all()


@pytest.mark.parametrize("E,k", [(96, 24), (160, 60)])
def test_reordered_choices_of_many_tokens(E, k):
    # every token's first order is put right by other lanes than those that wrote it
    T = 4096
    g = torch.Generator().manual_seed(k)
    l = (torch.randn(T, E, generator=g) * 1e-6).cuda()
    b = (0.25 + torch.randint(0, 2, (E,), generator=g).float() * 2.0 ** -23)
    ids, _ = moe.route_scored(l, k, bias=b.cuda())
    key = 0.5 * torch.tanh(0.5 * l.double()) + b.double().cuda()  # (1/2 less: exact to 1e-17)
    assert torch.equal(ids.long(), torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_a_nan_among_close_keys_stays_last(score):
    # as many experts as are left without it, close to one another: put in order by their 64-bit keys
    for E, k in ((20, 19), (64, 63), (96, 8)):
        l = torch.zeros(4, E)
        l[:, 5] = float("nan")
        l = l.cuda()
        b = torch.full((E,), 0.25)
        b[5] = 2.0
        if score == "sigmoid":
            ids, _ = moe.route_scored(l, k, bias=b.cuda())
            assert (ids == torch.tensor([e for e in range(E) if e != 5][:k], dtype=torch.int32).cuda()).all()
        else:  # every score is NaN: any k experts
            ids, _ = moe.route_scored(l, k, bias=b.cuda(), score=score)
            assert all(len(set(r)) == k and 0 <= min(r) and max(r) < E for r in ids.tolist())
