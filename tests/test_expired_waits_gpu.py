"""Expired waits of the 4-bit product and of the grouped GEMM, without a fault: one
stage's copy of one CTA is never issued (include/moe_testing.h) and the waits
give up after a millisecond.  Whichever roles and lanes give up first, the launch
ends with MOE_ERR_TIMEOUT, and the next call is right."""
import pytest
import torch

import indirect_expert_matmul_b200 as moe

pytestmark = pytest.mark.gpu


def _product(T, E, k, n_in, n_out, seed):
    g = torch.Generator().manual_seed(seed)
    b = torch.randint(0, 256, (E, n_out, n_in // 32, 17), generator=g, dtype=torch.uint8)
    b[..., 0] = torch.randint(118, 122, (E, n_out, n_in // 32), generator=g, dtype=torch.uint8)
    W = moe.weights_prepare(b.cuda(), E, n_out, n_in, wtype="mxfp4")
    x = torch.randn(T, n_in, generator=g).bfloat16().cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    return W, x, ids


def _recovers(ws, call, want):
    torch.cuda.synchronize()
    assert moe.lib().moe_workspace_init(ws.data_ptr(), None) == moe.OK
    got = call()
    assert moe.get_status(ws) == moe.OK
    assert torch.equal(got, want)


# one launch of the few-slot form, and the GEMM by pairs of CTAs
@pytest.mark.parametrize("T,E,k,n_in,n_out", [(3, 3, 2, 1600, 300), (150, 3, 2, 1600, 300), (40, 2, 1, 4096, 200)])
def test_stalls_of_every_kind_of_stage(T, E, k, n_in, n_out):
    W, x, ids = _product(T, E, k, n_in, n_out, T)
    ws = moe.workspace(T, k, E, n_in)

    def call():
        return moe.mul_mat_id_mx4(W, E, n_out, n_in, x, ids, ws=ws)

    want = call()
    assert moe.get_status(ws) == moe.OK
    seen = 0
    for cta in (0, 1, 2, 3):
        for stage in (0, 1, 3, 4, 6, 7, 9):
            moe.lib().moe_testing_stall(cta, stage, 1000)
            try:
                out = call()
                st = moe.get_status(ws)
            finally:
                moe.lib().moe_testing_stall(-1, 0, 0)
            if st == moe.OK:  # the CTA has no such stage
                assert torch.equal(out, want)
            else:
                assert st == moe.ERR_TIMEOUT
                seen += 1
            _recovers(ws, call, want)
    assert seen >= 4


NO_CTA = 1 << 20  # nothing is stalled: only the waits' limit is short


def _short_limits(ws, call, want, limits):
    """The waits of every role run out while what they wait for arrives."""
    late = 0
    for us in limits:
        for _ in range(4):
            moe.lib().moe_testing_stall(NO_CTA, 0, us)
            try:
                out = call()
                st = moe.get_status(ws)
            finally:
                moe.lib().moe_testing_stall(-1, 0, 0)
            if st == moe.OK:
                assert torch.equal(out, want)
            else:
                assert st == moe.ERR_TIMEOUT
                late += 1
        _recovers(ws, call, want)
    return late


# (a wait sleeps up to 20 us before it looks at its limit: long rows make longer waits)
LIMITS = [1, 2, 5, 10, 15, 20, 21, 22, 23, 24, 25, 30, 35, 40, 60]


@pytest.mark.parametrize("T,E,k,n_in,n_out", [(3, 30, 2, 1600, 300), (128, 60, 1, 9216, 2000), (900, 6, 2, 2880, 700),
                                              (300, 4, 2, 20480, 300), (500, 9, 2, 12288, 1200)])
def test_waits_that_run_out_while_copies_land(T, E, k, n_in, n_out):
    W, x, ids = _product(T, E, k, n_in, n_out, T)
    ws = moe.workspace(T, k, E, n_in)

    def call():
        return moe.mul_mat_id_mx4(W, E, n_out, n_in, x, ids, ws=ws)

    want = call()
    assert moe.get_status(ws) == moe.OK
    late = _short_limits(ws, call, want, LIMITS)
    assert late > 0 or n_in < 10000


@pytest.mark.parametrize("wtype,row", [("q8_0", 34), ("mxfp4", 17)])
def test_waits_of_the_grouped_gemm_that_run_out(wtype, row):
    T, E, k, n, ff = 600, 5, 3, 7168, 1024
    g = torch.Generator().manual_seed(3)

    def weights(n_out, n_in):
        b = torch.randint(0, 256, (E, n_out, n_in // 32, row), generator=g, dtype=torch.uint8)
        if wtype == "q8_0":
            b[..., 0], b[..., 1] = 0, 0x18  # scale 2^-9
        else:
            b[..., 0] = 118
        return moe.weights_prepare(b.cuda(), E, n_out, n_in, wtype=wtype)

    Wg, Wu, Wd = weights(ff, n), weights(ff, n), weights(n, ff)
    x = torch.randn(T, n, generator=g).bfloat16().cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    ws = moe.workspace(T, k, E, n, ff)

    def call():
        return moe.ffn(Wg, Wu, Wd, E, n, ff, x, ids, ws=ws, wtype=wtype)[0]

    want = call()
    assert moe.get_status(ws) == moe.OK
    assert _short_limits(ws, call, want, LIMITS) > 0
