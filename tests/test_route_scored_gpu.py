"""moe_route_scored and its gradient against a 64-bit implementation: sigmoid and
softmax scores, balance bias, groups, ties, -inf logits, odd sizes, strided rows
and half-precision logits; ids exactly, weights and gradients within float32
bounds; gradients also against differences of the forward rule."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_b200 as moe
from tests import routed_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _logits(T, E, dtype, seed, std=1.5, pad=0):
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn(T, E + pad, generator=g) * std).to(DT[dtype]).cuda()
    return wide[:, :E]


def _bias(E, seed):
    return (torch.randn(E, generator=torch.Generator().manual_seed(seed)) * 0.05).cuda()


def _check(l, k, bias, **kw):
    opt = dict(score="sigmoid", n_groups=1, topk_groups=1, group_score="max", normalize=True, scale=1.0)
    opt.update(kw)
    ids, w = moe.route_scored(l, k, bias=bias, **opt)
    r_ids, r_w, tol = ref.route(l.double().cpu().numpy(), k, None if bias is None else bias.double().cpu().numpy(),
                                **opt)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    err = np.abs(w.double().cpu().numpy() - r_w)
    assert (err <= tol).all(), float((err / tol).max())
    ids2, w2 = moe.route_scored(l, k, bias=bias, **opt)
    assert torch.equal(ids, ids2) and torch.equal(w.view(torch.int32), w2.view(torch.int32))
    return ids, w


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,groups,dtype", [
    (1, 256, 8, (8, 4, "top2"), "f32"), (65, 256, 8, (8, 4, "max"), "f32"), (33, 160, 6, (8, 3, "top2"), "bf16"),
    (7, 60, 4, (12, 5, "top2"), "f16"), (5, 1024, 16, (32, 7, "top2"), "f32"), (9, 7, 7, (1, 1, "max"), "f32"),
    (3, 1, 1, (1, 1, "max"), "bf16"), (17, 100, 40, (2, 1, "top2"), "f32"), (6, 31, 3, (31, 5, "max"), "f32"),
    (4, 300, 10, (4, 4, "top2"), "bf16"), (5, 512, 9, (16, 15, "top2"), "f16"), (2, 66, 40, (3, 2, "max"), "f32")])
def test_route_scored(score, normalize, T, E, k, groups, dtype):
    G, top, gs = groups
    l = _logits(T, E, dtype, T * E + k)
    for bias in (None, _bias(E, E)):
        _check(l, k, bias, score=score, normalize=normalize, n_groups=G, topk_groups=top, group_score=gs, scale=2.5)


@pytest.mark.parametrize("pad", [1, 16])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_strided_rows(pad, dtype):
    l = _logits(19, 96, dtype, 5, pad=pad)
    assert not l.is_contiguous()
    _check(l, 6, _bias(96, 1), n_groups=4, topk_groups=2, group_score="top2")


def test_many_tokens_ids_exact():
    # close keys occur among 16384 tokens; the choice must be the 64-bit one in each
    _check(_logits(16384, 128, "f32", 77), 8, _bias(128, 3), n_groups=8, topk_groups=4, group_score="top2")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_keys_closer_than_float32(score):
    # scores saturated near one, or almost uniform, and biases that differ in the last place
    T, E = 64, 64
    g = torch.Generator().manual_seed(9)
    l = (torch.rand(T, E, generator=g) * 1e-6 + (12.0 if score == "sigmoid" else 0.0)).cuda()
    bias = (0.05 + torch.randint(0, 4, (E,), generator=g).float() * 2.0 ** -28).cuda()
    _check(l, 8, bias, score=score, n_groups=8, topk_groups=3, group_score="top2")
    _check(l, 8, bias, score=score, n_groups=8, topk_groups=3, group_score="max")
    _check(l, 8, bias, score=score)
    _check(l, 8, None, score=score, n_groups=8, topk_groups=3, group_score="top2")


def test_group_sums_of_large_opposite_biases():
    # a group's two largest keys are s + 64 and s' - 64: their sum is a sum of two
    # scores that a float key cannot hold to better than 2^-18
    T, G, m = 64, 8, 16
    g = torch.Generator().manual_seed(4)
    bias = torch.full((G, m), -1000.0)
    bias[:, 3], bias[:, 9] = 64.0, -64.0
    bias = bias.reshape(-1).cuda()
    l = (torch.randn(T, G * m, generator=g) * 1e-5).cuda()  # sums of scores a few 1e-6 apart
    for size in (m, 12):  # groups that are whole lanes, and groups that are not
        E = G * size
        b, x = bias.view(G, m)[:, :size].reshape(-1).contiguous(), l.view(T, G, m)[:, :, :size].reshape(T, E).contiguous()
        _check(x, 2, b, n_groups=G, topk_groups=3, group_score="top2")


def test_exact_ties_take_the_lower_index():
    l = torch.zeros(3, 96).cuda()
    l[1, 40:] = 1.0
    l[2, ::7] = -1.0
    for bias in (None, torch.zeros(96).cuda()):
        ids, _ = _check(l, 8, bias)
        assert ids[0].tolist() == list(range(8)) and ids[1].tolist() == list(range(40, 48))
        _check(l, 8, bias, n_groups=6, topk_groups=2, group_score="top2")
        _check(l, 8, bias, score="softmax", n_groups=6, topk_groups=2)


def test_masked_experts_and_empty_rows():
    inf = float("inf")
    l = _logits(6, 64, "f32", 3)
    l[1, 8:] = -inf         # 8 experts left, k = 8
    l[2, 4:] = -inf         # fewer left than k
    l[3] = -inf             # none left
    l[4] = torch.finfo(torch.float32).min
    l[5, ::2] = torch.finfo(torch.float32).min
    for score in ("sigmoid", "softmax"):
        for normalize in (True, False):
            for bias in (None, _bias(64, 4)):
                ids, w = moe.route_scored(l, 8, bias=bias, score=score, normalize=normalize)
                r_ids, r_w, tol = ref.route(l.double().cpu().numpy(), 8,
                                            None if bias is None else bias.double().cpu().numpy(), score, 1, 1, "max",
                                            normalize, 1.0)
                assert torch.isfinite(w).all()
                w = w.double().cpu().numpy()
                rows = [0, 1, 2, 3, 4]
                assert np.array_equal(ids.cpu().numpy()[rows], r_ids[rows])
                assert (np.abs(w - r_w)[:4] <= tol[:4]).all()
                assert (w[3] == 0).all()
                if score == "sigmoid" and not normalize:
                    assert (w[4] == 0).all()
                elif bias is None:  # equal logits at the type's lowest value are equal scores
                    assert np.abs(w[4] - (1 / 8 if normalize else 1 / 64)).max() <= 128 * ref.U
                assert len(set(ids[5].tolist())) == 8


def test_nan_and_inf_logits_give_valid_ids():
    l = _logits(4, 96, "f32", 8)
    l[0, 5] = float("nan")
    l[1] = float("nan")
    l[2, 3] = float("inf")
    l[3, :50] = float("nan")
    for kw in (dict(), dict(score="softmax"), dict(n_groups=6, topk_groups=2, group_score="top2")):
        for bias in (None, _bias(96, 2)):
            ids, _ = moe.route_scored(l, 8, bias=bias, **kw)
            for row in ids.tolist():
                assert len(set(row)) == 8 and min(row) >= 0 and max(row) < 96
                if "n_groups" in kw:
                    assert len({e // 16 for e in row}) <= 2
    assert 5 not in moe.route_scored(l, 8)[0][0].tolist()


@pytest.mark.parametrize("shift", [-90.0, -300.0, 60.0])
def test_normalised_weights_far_from_zero(shift):
    l = _logits(8, 64, "f32", 21) + shift
    for score in ("sigmoid", "softmax"):
        ids, w = moe.route_scored(l, 6, score=score)
        s = w.double().sum(-1)
        assert torch.isfinite(w).all() and (s - 1).abs().max().item() <= 32 * ref.U
        # the choice: sigmoids that a float cannot tell apart still follow their logits
        order = torch.sort(l, dim=-1, descending=True, stable=True).indices[:, :6]
        assert torch.equal(ids.long(), order)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,dtype,pad", [(1, 256, 8, "f32", 0), (67, 256, 8, "bf16", 0), (9, 61, 5, "f16", 3),
                                             (5, 1024, 40, "f32", 0), (3, 1, 1, "f32", 0), (300, 128, 4, "bf16", 16),
                                             (4, 33, 33, "f32", 0)])
def test_backward(score, normalize, T, E, k, dtype, pad):
    l = _logits(T, E, dtype, T + E, pad=pad)
    ids, _ = moe.route_scored(l, k, score=score, normalize=normalize, bias=_bias(E, 7))
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(T)).cuda()
    d = moe.route_scored_backward(l, ids, dw, score=score, normalize=normalize, scale=2.5)
    assert d.dtype == l.dtype and tuple(d.shape) == (T, E)
    half = torch.finfo(DT[dtype]).eps / 2
    r, tol = ref.route_grad(l.double().cpu().numpy(), ids.cpu().numpy(), dw.double().cpu().numpy(), score, normalize,
                            2.5, half)
    err = np.abs(d.double().cpu().numpy() - r)
    assert (err <= tol).all(), float((err / tol).max())
    d2 = moe.route_scored_backward(l, ids, dw, score=score, normalize=normalize, scale=2.5)
    assert torch.equal(d, d2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [True, False])
def test_backward_against_differences(score, normalize):
    T, E, k, h = 5, 24, 4, 1e-5
    l = _logits(T, E, "f32", 31)
    ids, _ = moe.route_scored(l, k, score=score, normalize=normalize)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    d = moe.route_scored_backward(l, ids, dw, score=score, normalize=normalize, scale=1.7).double().cpu().numpy()
    ln, idn, g = l.double().cpu().numpy(), ids.cpu().numpy(), dw.double().cpu().numpy()

    def loss(x):
        s = np.take_along_axis(ref.scores(x, score), idn, 1)
        w = 1.7 * (s / s.sum(1, keepdims=True) if normalize else s)
        return (w * g).sum(1)

    for e in range(E):
        up, dn = ln.copy(), ln.copy()
        up[:, e] += h
        dn[:, e] -= h
        fd = (loss(up) - loss(dn)) / (2 * h)
        # the difference quotient is off by h^2/6 times a third derivative of at most ~40; float32: 1e-5
        assert np.abs(fd - d[:, e]).max() <= 40 * h * h + 1e-5


def test_backward_repeated_unused_and_masked_slots():
    l = _logits(4, 64, "f32", 12)
    l[2, 8:] = -float("inf")
    l[3] = -float("inf")
    ids = torch.tensor([[3, 3, 5, 3], [-1, 7, 64, 9], [1, 20, 2, 40], [0, 1, 2, 3]], dtype=torch.int32).cuda()
    dw = torch.randn(4, 4, generator=torch.Generator().manual_seed(2)).cuda()
    for score in ("sigmoid", "softmax"):
        for normalize in (True, False):
            d = moe.route_scored_backward(l, ids, dw, score=score, normalize=normalize)
            r, tol = ref.route_grad(l.double().cpu().numpy(), ids.cpu().numpy(), dw.double().cpu().numpy(), score,
                                    normalize, 1.0, ref.U)
            d = d.double().cpu().numpy()
            assert np.isfinite(d).all()
            assert (np.abs(d - r) <= tol).all()
            assert (d[3] == 0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,dtype,pad", [(4737, 128, 4, "bf16", 16), (4741, 33, 33, "f32", 0),
                                             (5003, 100, 17, "f16", 1), (4801, 1, 1, "f32", 0), (4999, 31, 9, "bf16", 3)])
def test_backward_of_many_tokens(score, normalize, T, E, k, dtype, pad):
    """Up to 128 experts and above 4736 tokens half a warp has a token."""
    l = _logits(T, E, dtype, T + E, pad=pad)
    l[1, 1:] = -float("inf")
    l[T - 1] = -float("inf")
    g = torch.Generator().manual_seed(T)
    ids = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32)
    ids[::3, 0] = ids[::3, k - 1]  # twice in a row
    ids[::5, k // 2] = -1
    ids[1::5, k // 2] = E
    ids, dw = ids.cuda(), torch.randn(T, k, generator=g).cuda()
    d = moe.route_scored_backward(l, ids, dw, score=score, normalize=normalize, scale=2.5)
    half = torch.finfo(DT[dtype]).eps / 2
    r, tol = ref.route_grad(l.double().cpu().numpy(), ids.cpu().numpy(), dw.double().cpu().numpy(), score, normalize,
                            2.5, half)
    err = np.abs(d.double().cpu().numpy() - r)
    assert (err <= tol).all(), float((err / tol).max())
    # the same rows by themselves, a warp each, are the same up to their roundings
    few = moe.route_scored_backward(l[:70], ids[:70].contiguous(), dw[:70].contiguous(), score=score,
                                    normalize=normalize, scale=2.5)
    assert (np.abs(few.double().cpu().numpy() - r[:70]) <= tol[:70]).all()


def test_rows_behind_the_last_token_are_left_alone():
    l = _logits(5, 64, "f32", 2)
    ids = torch.full((8, 4), -7, dtype=torch.int32).cuda()
    w = torch.full((8, 4), -7.0).cuda()
    moe.route_scored(l, 4, ids=ids, weights=w)
    assert (ids[5:] == -7).all() and (w[5:] == -7).all() and (ids[:5] >= 0).all()
    out = torch.full((8, 64), -7.0).cuda()
    moe.route_scored_backward(l, ids[:5], w[:5].contiguous(), out=out)
    assert (out[5:] == -7).all()
    e_ids, e_w = moe.route_scored(l[:0], 4)
    assert e_ids.shape == (0, 4) and e_w.shape == (0, 4)
    assert moe.route_scored_backward(l[:0], e_ids, e_w).shape == (0, 64)


def test_graph_replay_and_side_stream():
    l = _logits(33, 256, "f32", 4)
    b = _bias(256, 4)
    dw = torch.randn(33, 8, generator=torch.Generator().manual_seed(5)).cuda()
    kw = dict(score="sigmoid", normalize=True, scale=2.5)
    ids, w = moe.route_scored(l, 8, bias=b, n_groups=8, topk_groups=4, group_score="top2", **kw)
    d = moe.route_scored_backward(l, ids, dw, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids2, w2, d2 = torch.empty_like(ids), torch.empty_like(w), torch.empty_like(d)
    with torch.cuda.stream(side):
        moe.route_scored(l, 8, bias=b, n_groups=8, topk_groups=4, group_score="top2", ids=ids2, weights=w2, **kw)
        moe.route_scored_backward(l, ids2, dw, out=d2, **kw)
    side.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(d, d2)
    ids2.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.route_scored(l, 8, bias=b, n_groups=8, topk_groups=4, group_score="top2", ids=ids2, weights=w2, **kw)
        moe.route_scored_backward(l, ids2, dw, out=d2, **kw)
    new = _logits(33, 256, "f32", 99)
    l.copy_(new)
    g.replay()
    torch.cuda.synchronize()
    ids, w = moe.route_scored(new, 8, bias=b, n_groups=8, topk_groups=4, group_score="top2", **kw)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    assert torch.equal(moe.route_scored_backward(new, ids, dw, **kw), d2)
