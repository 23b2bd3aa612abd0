"""moe_combine_backward against a 64-bit implementation: dweights within the
float32 bound of the sum, ddst exactly the float product, over vector and
scalar layouts, one slot to many, in place, without ddst."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_b200 as moe
from tests import routed_ref as ref

pytestmark = pytest.mark.gpu


def _inputs(T, k, n, seed=0):
    g = torch.Generator().manual_seed(seed + T * k + n)
    return (torch.randn(T, n, generator=g).cuda(), torch.randn(T, k, n, generator=g).cuda(),
            torch.randn(T, k, generator=g).cuda())


def _check(dy, dst, w, dw, dd, dst_in=None):
    r_dw, tol, _ = ref.combine_grad(dy.cpu().numpy(), (dst if dst_in is None else dst_in).cpu().numpy(),
                                    w.cpu().numpy())
    err = np.abs(dw.double().cpu().numpy() - r_dw)
    assert (err <= tol).all(), float((err / tol).max())
    if dd is not None:
        assert torch.equal(dd, w[:, :, None] * dy[:, None, :])


@pytest.mark.parametrize("T,k,n", [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (5, 6, 1001), (64, 6, 2048), (17, 9, 4100),
                                   (2, 40, 96), (300, 4, 2880), (9, 8, 7168), (1, 1, 20000), (2, 3, 16388),
                                   (700, 1, 33), (2, 20, 7168)])
def test_combine_backward(T, k, n):
    dy, dst, w = _inputs(T, k, n)
    dw, dd = moe.combine_backward(dy, dst, w)
    _check(dy, dst, w, dw, dd)
    dw2, none = moe.combine_backward(dy, dst, w, need_ddst=False)
    assert none is None and torch.equal(dw, dw2)


def test_in_place_and_reruns():
    dy, dst, w = _inputs(40, 6, 1408)
    dw, dd = moe.combine_backward(dy, dst, w)
    keep = dst.clone()
    dw2, dd2 = moe.combine_backward(dy, dst, w, ddst=dst)
    assert dd2 is dst and torch.equal(dw, dw2) and torch.equal(dd, dst)
    _check(dy, dst, w, dw2, dd2, keep)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_buffers_take_the_scalar_path(off):
    T, k, n = 5, 3, 256
    dy, dst, w = _inputs(T, k, n)
    big = torch.full((T * k * n + 4,), -7.0).cuda()
    view = big[off:off + T * k * n].view(T, k, n)
    dw, _ = moe.combine_backward(dy, dst, w, ddst=view)
    _check(dy, dst, w, dw, view)
    assert (big[:off] == -7).all() and (big[off + T * k * n:] == -7).all()
    src = torch.empty(T * k * n + 4).cuda()[off:off + T * k * n].view(T, k, n)
    src.copy_(dst)
    dw2, _ = moe.combine_backward(dy, src, w)
    _check(dy, dst, w, dw2, None)


def test_gradient_against_differences():
    T, k, n = 2, 3, 5
    dy, dst, w = _inputs(T, k, n)
    dw, dd = (t.double().cpu().numpy() for t in moe.combine_backward(dy, dst, w))
    dyn, dn, wn = (t.double().cpu().numpy() for t in (dy, dst, w))
    loss = lambda d, v: (np.einsum("tk,tkn->tn", v, d) * dyn).sum()  # linear in each: differences are exact but for rounding
    for t in range(T):
        for s in range(k):
            v = wn.copy()
            v[t, s] += 0.5
            assert abs((loss(dn, v) - loss(dn, wn)) / 0.5 - dw[t, s]) < 1e-5
            for j in range(n):
                d = dn.copy()
                d[t, s, j] += 0.5
                assert abs((loss(d, wn) - loss(dn, wn)) / 0.5 - dd[t, s, j]) < 1e-5


def test_no_tokens_and_rows_behind():
    dy, dst, w = _inputs(3, 2, 64)
    out = torch.full((5, 2), -7.0).cuda()
    moe.combine_backward(dy, dst, w, need_ddst=False, dweights=out)
    assert (out[3:] == -7).all()
    dw, dd = moe.combine_backward(dy[:0], dst[:0], w[:0])
    assert dw.shape == (0, 2) and dd.shape == (0, 2, 64)
