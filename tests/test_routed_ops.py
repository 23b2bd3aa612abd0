"""Host side of the scored router, the gradients, MXFP4 quantisation and the
4-bit product: argument checks that need no GPU, and the 64-bit test
implementations against hand-worked values."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_b200 as moe
from tests import routed_ref as ref

P = 4096  # an aligned non-null address: every call below is refused before it is used


def _route(T=4, E=64, k=8, ld=None, lt=2, score=1, groups=(8, 4, 2), logits=P, bias=P, ids=P, w=P):
    return moe.lib().moe_route_scored(logits, lt, E if ld is None else ld, bias, T, E, k, score, *groups, 1, 1.0, ids,
                                      w, None)


def _bwd(T=4, E=64, k=8, ld=None, lt=2, score=1, logits=P, ids=P, dw=P, out=P):
    return moe.lib().moe_route_scored_backward(logits, lt, E if ld is None else ld, ids, dw, T, E, k, score, 1, 1.0,
                                               out, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(k=0), dict(k=65), dict(E=0), dict(ld=63), dict(lt=3), dict(lt=-1), dict(score=2),
    dict(groups=(0, 1, 1)), dict(groups=(7, 4, 1)), dict(groups=(8, 0, 1)), dict(groups=(8, 9, 1)),
    dict(groups=(8, 4, 0)), dict(groups=(8, 4, 3)), dict(groups=(8, 1, 1), k=9), dict(groups=(64, 64, 2), E=64),
    dict(logits=None), dict(ids=None), dict(w=None), dict(logits=P + 2), dict(logits=P + 1, lt=0), dict(bias=P + 2),
    dict(ids=P + 1), dict(w=P + 2)])
def test_route_scored_refusals(kw):
    assert _route(**kw) in (moe.ERR_INVALID, moe.ERR_RANGE)
    if kw != dict(groups=(64, 64, 2), E=64):
        assert _route(**kw) == moe.ERR_INVALID


@pytest.mark.parametrize("kw", [dict(T=1 << 22), dict(E=1088, groups=(1, 1, 1)), dict(groups=(64, 64, 1)),
                                dict(ld=1 << 40)])
def test_route_scored_range(kw):
    assert _route(**kw) == moe.ERR_RANGE


@pytest.mark.parametrize("kw", [dict(T=-1), dict(k=0), dict(k=65), dict(ld=63), dict(lt=3), dict(score=-1),
                                dict(logits=None), dict(ids=None), dict(dw=None), dict(out=None), dict(out=P + 2),
                                dict(ids=P + 2), dict(dw=P + 1)])
def test_route_scored_backward_refusals(kw):
    assert _bwd(**kw) == moe.ERR_INVALID


def test_backward_ranges_and_empty_calls():
    assert _bwd(T=1 << 22) == moe.ERR_RANGE and _bwd(E=1025) == moe.ERR_RANGE and _bwd(ld=1 << 40) == moe.ERR_RANGE
    assert _route(T=0, logits=None, ids=None, w=None) == moe.OK
    assert _bwd(T=0, logits=None, ids=None, dw=None, out=None) == moe.OK
    L = moe.lib()
    assert L.moe_combine_backward(None, None, None, 0, 2, 8, None, None, None) == moe.OK
    assert L.moe_mxfp4_quantize(None, 0, 32, 0, 32, None, None, None) == moe.OK
    assert L.moe_mul_mat_id_mx4(P, 4, 8, 64, None, 0, None, 0, 1, 0, None, P, None) == moe.OK


def test_combine_backward_refusals():
    f = moe.lib().moe_combine_backward
    for a in [(P, P, P, -1, 2, 8, P, P), (P, P, P, 4, 0, 8, P, P), (P, P, P, 4, 2, 0, P, P),
              (None, P, P, 4, 2, 8, P, P), (P, None, P, 4, 2, 8, P, P), (P, P, None, 4, 2, 8, P, P),
              (P, P, P, 4, 2, 8, None, P), (P + 2, P, P, 4, 2, 8, P, P), (P, P, P, 4, 2, 8, P, P + 1)]:
        assert f(*a, None) == moe.ERR_INVALID
    for a in [(1 << 22, 2, 8), (4, 1024, 8), (4, 2, 1 << 31)]:
        assert f(P, P, P, *a, P, P, None) == moe.ERR_RANGE


def test_mxfp4_quantize_refusals():
    f = moe.lib().moe_mxfp4_quantize
    for a in [(P, 3, 64, 4, 64, P, None), (P, 0, 63, 4, 64, P, None), (P, 0, 64, -1, 64, P, None),
              (P, 0, 64, 4, 48, P, None), (P, 0, 64, 4, 0, P, None), (None, 0, 64, 4, 64, P, None),
              (P, 0, 64, 4, 64, None, None), (P + 1, 0, 64, 4, 64, P, None), (P + 2, 2, 64, 4, 64, P, None),
              (P, 0, 64, 4, 64, P, P + 8)]:
        assert f(*a, None) == moe.ERR_INVALID
    for a in [(64, 1 << 31, 64), (1 << 40, 4, 64)]:
        assert f(P, 0, *a, P, None, None) == moe.ERR_RANGE


def test_mx4_product_refusals():
    f = moe.lib().moe_mul_mat_id_mx4
    good = dict(W=P, E=4, n_out=8, n_in=64, x=P, xt=0, ids=P, T=2, k=1, mode=0, dst=P, ws=P)

    def call(**kw):
        a = dict(good, **kw)
        return f(a["W"], a["E"], a["n_out"], a["n_in"], a["x"], a["xt"], a["ids"], a["T"], a["k"], a["mode"], a["dst"],
                 a["ws"], None)

    for kw in [dict(W=None), dict(W=P + 128), dict(E=0), dict(n_out=0), dict(n_in=48), dict(n_in=0), dict(x=None),
               dict(x=P + 8), dict(xt=3), dict(ids=None), dict(T=-1), dict(k=0), dict(mode=2), dict(dst=None),
               dict(dst=P + 4), dict(ws=None), dict(ws=P + 128)]:
        assert call(**kw) == moe.ERR_INVALID, kw
    for kw in [dict(k=5), dict(T=1 << 22), dict(k=1024, E=2000), dict(E=16385), dict(T=(1 << 22) - 1, k=1000, E=1000)]:
        assert call(**kw) == moe.ERR_RANGE, kw


def test_binding_refuses_wrong_tensors():
    cpu = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moe.route_scored(cpu, 4)
    with pytest.raises(ValueError):
        moe.route_scored(cpu.double(), 4)
    with pytest.raises(ValueError):
        moe.route_scored(torch.zeros(64), 4)
    with pytest.raises(ValueError):
        moe.mxfp4_quantize(cpu)
    with pytest.raises(ValueError):
        moe.combine_backward(cpu, cpu, cpu)
    with pytest.raises(ValueError):
        moe.mul_mat_id_mx4(cpu, 1, 1, 32, cpu, cpu)


def test_binding_checks_layout(monkeypatch):
    monkeypatch.setattr(moe, "_gpu", lambda t, name: None)  # no GPU here: accept host tensors as device ones
    assert moe._rows(torch.zeros(3, 40)[:, :32], "x") == (3, 32, 40)
    assert moe._rows(torch.zeros(1, 40)[:, :32], "x")[:2] == (1, 32)
    assert moe._rows(torch.zeros(2, 3, 32), "x") == (6, 32, 32)
    assert moe._rows(torch.zeros(0, 32), "x")[:2] == (0, 32)
    for bad in (torch.zeros(32, 3).t(), torch.zeros(2, 3, 40)[..., :32], torch.zeros(1, 32).expand(4, 32)):
        with pytest.raises(ValueError):
            moe._rows(bad, "x")
    for x in (torch.zeros(4, 48), torch.zeros(4, 0), torch.zeros(4, 32).double()):
        with pytest.raises(ValueError):
            moe.mxfp4_quantize(x)
    l = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="holds"):
        moe.route_scored(l, 2, ids=torch.zeros(4, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        moe.route_scored_backward(l, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2))


# ------------------------------------------------- the test implementations
def test_reference_rounding_by_hand():
    x = np.zeros((1, 32))
    x[0, :12] = [6.0, 5.0, 2.5, -2.51, 0.25, 0.26, 0.75, 1.75, 3.5, 7.0, -0.0, -1.25]
    v, X, code = ref.mx_round(x)
    assert X[0, 0] == 127  # floor(log2 7) - 2 = 0
    assert v[0, :12].tolist() == [6, 4, 2, -3, 0, 0.5, 1, 2, 4, 6, 0, -1]
    assert code[0, 0, :12].tolist() == [7, 6, 4, 13, 0, 1, 2, 4, 6, 7, 8, 10]
    b = ref.mx_blocks(X, code)
    assert b[0, 0, 0] == 127 and b[0, 0, 1] == 7 and np.array_equal(ref.mx_weights(b), v)


def test_reference_router_by_hand():
    l = np.log(np.array([[1.0, 3.0, 1.0, 1 / 3, 9.0, 1 / 9]]))  # sigmoids 1/2 3/4 1/2 1/4 9/10 1/10
    ids, w, _ = ref.route(l, 2, None, "sigmoid", 1, 1, "max", False, 1.0)
    assert ids.tolist() == [[4, 1]] and np.allclose(w, [[0.9, 0.75]])
    # groups {0,1} {2,3} {4,5}: sums of two 1.25, 0.75, 1.0; the best group alone
    ids, w, _ = ref.route(l, 2, None, "sigmoid", 3, 1, "top2", True, 2.0)
    assert ids.tolist() == [[1, 0]] and np.allclose(w, [[1.2, 0.8]])
    ids, _, _ = ref.route(l, 2, np.array([0, 0, 0, 0, -1.0, 0]), "sigmoid", 1, 1, "max", True, 1.0)
    assert ids.tolist() == [[1, 0]]
    p = ref.scores(np.array([[0.0, 0.0, -np.inf]]), "softmax")
    assert p.tolist() == [[0.5, 0.5, 0.0]]


def test_reference_gradient_by_differences():
    rng = np.random.default_rng(0)
    l, ids, g, h = rng.normal(size=(2, 6)), np.array([[4, 1, 0], [2, 5, 3]]), rng.normal(size=(2, 3)), 1e-6
    for score in ("sigmoid", "softmax"):
        for normalize in (True, False):
            d, _ = ref.route_grad(l, ids, g, score, normalize, 1.5, ref.U)

            def loss(x):
                s = np.take_along_axis(ref.scores(x, score), ids, 1)
                return 1.5 * (g * (s / s.sum(1, keepdims=True) if normalize else s)).sum()

            for t in range(2):
                for e in range(6):
                    a, b = l.copy(), l.copy()
                    a[t, e] += h
                    b[t, e] -= h
                    assert abs((loss(a) - loss(b)) / (2 * h) - d[t, e]) < 1e-8


def test_slots_that_leave_32_bits_on_the_way_are_refused():
    # 2147483136 and a little fewer slots: positions padded by expert, or stepped past the last slot, pass 2^31
    L, nul = moe.lib(), None
    T = (1 << 22) - 1
    for k, E, tokens in ((512, 512, T), (512, 1024, T), (512, 512, T - 16), (1023, 1023, (1 << 31) // 1023)):
        assert tokens * k < 1 << 31
        assert L.moe_row_ids(nul, tokens, k, E, 0, nul, nul, nul, nul, nul) == moe.ERR_RANGE
        assert L.moe_mul_mat_id(nul, E, 8, 64, nul, 0, nul, tokens, k, 0, nul, nul, nul) == moe.ERR_RANGE
        assert L.moe_ffn(nul, nul, nul, E, 64, 64, nul, nul, nul, 0, nul, 0, nul, tokens, k, nul, nul, nul,
                         nul) == moe.ERR_RANGE
        assert L.moe_mul_mat_id_mx4(nul, E, 8, 64, nul, 0, nul, tokens, k, 0, nul, nul, nul) == moe.ERR_RANGE
    assert L.moe_row_ids(nul, T, 511, 1024, 0, nul, nul, nul, nul, nul) == moe.ERR_INVALID  # (null pointers)
    assert L.moe_mul_mat_id_mx4(nul, 1024, 8, 64, nul, 0, nul, T, 511, 0, nul, nul, nul) == moe.ERR_INVALID


@pytest.mark.parametrize("n_in", [32, 64, 96, 7168])
def test_workspace_holds_what_the_products_use(n_in):
    # header, slot and expert tables, 16-bit rows by 64 values, and a factor a row (for up to 64 values the
    # 4-bit product's 8 scale bytes take its place; beyond, they lie behind its codes)
    T, k, E = 4096, 8, 256
    up = lambda v: (v + 255) // 256 * 256
    rows = T * k + 8 * E + 32
    size = 256 + 3 * up(T * k * 4) + 4 * up((E + 1) * 4) + up((2 * 64 * E + E) * 4)
    size += up(rows * ((n_in + 63) // 64) * 128)
    size += up(rows * (8 if n_in <= 64 else 4))
    assert moe.workspace_size(T, k, E, n_in) == size
    planes, scale_rows = (n_in + 255) // 256, (rows + 3) // 4 * 4
    if n_in > 64:
        assert planes * (rows * 128 + scale_rows * 8) <= rows * ((n_in + 63) // 64) * 128
