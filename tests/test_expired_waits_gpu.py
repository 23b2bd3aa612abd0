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
