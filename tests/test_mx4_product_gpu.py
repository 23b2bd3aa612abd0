"""moe_mul_mat_id_mx4 against a 64-bit implementation.  The operands are exact
(x is rounded to MXFP4 by a rule without tolerance), so only the float32 sum
remains: n_in additions, each off by at most one unit in the last place of a
partial sum, which is at most the sum of the terms' magnitudes - a bound of
n_in * 2^-23 * sum |w x|."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_b200 as moe
from tests import routed_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _weights(E, n_out, n_in, seed, lo=117, hi=123):
    g = torch.Generator().manual_seed(seed)
    b = torch.randint(0, 256, (E, n_out, n_in // 32, 17), generator=g, dtype=torch.uint8)
    b[..., 0] = torch.randint(lo, hi, (E, n_out, n_in // 32), generator=g, dtype=torch.uint8)
    return b


def _ids(T, k, E, seed, only=None):
    g = torch.Generator().manual_seed(seed)
    pool = torch.arange(E) if only is None else torch.tensor(only)
    return torch.stack([pool[torch.randperm(len(pool), generator=g)[:k]] for _ in range(T)]).int()


def _run(blocks, x, ids, mode, **kw):
    E, n_out, nb, _ = blocks.shape
    W = moe.weights_prepare(blocks.cuda(), E, n_out, nb * 32, wtype="mxfp4")
    return moe.mul_mat_id_mx4(W, E, n_out, nb * 32, x, ids.cuda(), mode=mode, **kw)


def _check(blocks, x, ids, mode):
    dst = _run(blocks, x, ids, mode)
    out, mag = ref.mx_product(blocks.numpy(), x.double().cpu().numpy(), ids.numpy(), mode == "per_slot")
    err = np.abs(dst.double().cpu().numpy() - out)
    n_in = blocks.shape[2] * 32
    tol = n_in * 2.0 ** -23 * mag
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(~(err <= tol))[:4].tolist())
    dst2 = _run(blocks, x, ids, mode)
    assert torch.equal(dst.view(torch.int32), dst2.view(torch.int32))
    return dst


@pytest.mark.parametrize("mode", ["broadcast", "per_slot"])
@pytest.mark.parametrize("T,E,k,n_in,n_out,dtype", [
    (1, 1, 1, 32, 1, "f32"), (1, 8, 2, 32, 16, "bf16"), (1, 16, 8, 2048, 512, "bf16"), (4, 32, 8, 256, 130, "f16"),
    (3, 4, 2, 96, 33, "f32"), (8, 8, 4, 352, 144, "bf16"), (40, 4, 2, 512, 260, "bf16"), (65, 3, 3, 160, 129, "f32"),
    (300, 2, 1, 288, 128, "f16"), (257, 5, 4, 1408, 96, "bf16"), (130, 60, 6, 128, 200, "f32"),
    (17, 300, 10, 64, 40, "bf16")])
def test_product(mode, T, E, k, n_in, n_out, dtype):
    blocks = _weights(E, n_out, n_in, n_in + n_out)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T if mode == "broadcast" else T * k, n_in, generator=g).to(DT[dtype]).cuda()
    _check(blocks, x, _ids(T, k, E, T + E), mode)


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("n_out", [16, 47, 48, 80, 112, 128, 144, 208, 256, 272, 368])
def test_every_kind_of_last_tile(T, n_out):
    # last tiles of 16 to 112 rows (32-row sub-blocks, a 16-row one, both), odd and even tile counts
    blocks = _weights(3, n_out, 192, n_out)
    x = torch.randn(T, 192, generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
    _check(blocks, x, _ids(T, 2, 3, n_out), "broadcast")


@pytest.mark.parametrize("n_in", [32, 64, 96, 128, 160, 224, 256, 288, 480, 512, 544, 1056])
def test_every_kind_of_last_stage(n_in):
    blocks = _weights(2, 40, n_in, n_in)
    for T in (2, 140):
        x = torch.randn(T, n_in, generator=torch.Generator().manual_seed(n_in)).cuda()
        _check(blocks, x, _ids(T, 2, 2, n_in), "broadcast")


@pytest.mark.parametrize("T,E,k", [(40, 300, 10), (33, 1100, 9), (20, 1100, 8), (300, 1024, 2)])
def test_many_experts(T, E, k):
    # tables read from memory (more than 256 experts) and the general row-id pass (more than 1024)
    blocks = _weights(E, 24, 64, E)
    x = torch.randn(T, 64, generator=torch.Generator().manual_seed(E)).bfloat16().cuda()
    _check(blocks, x, _ids(T, k, E, T), "broadcast")


@pytest.mark.parametrize("mode,T,k", [("broadcast", 11000, 3), ("per_slot", 16400, 2)])
def test_more_slots_than_a_cta_counts(mode, T, k):
    blocks = _weights(7, 17, 64, T)
    x = torch.randn(T if mode == "broadcast" else T * k, 64, generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
    _check(blocks, x, _ids(T, k, 7, T), mode)


@pytest.mark.parametrize("T,n_in", [(2, 9216), (2, 9248), (1, 12320)])
def test_long_rows(T, n_in):
    # the longest that the one-launch form holds in shared memory, and past it
    blocks = _weights(2, 20, n_in, n_in)
    x = torch.randn(T, n_in, generator=torch.Generator().manual_seed(n_in)).bfloat16().cuda()
    _check(blocks, x, _ids(T, 2, 2, 1), "broadcast")


@pytest.mark.parametrize("S", [31, 32, 33, 255, 256, 257])
def test_slot_counts_at_the_borders_of_the_forms(S):
    blocks = _weights(5, 36, 96, S)
    x = torch.randn(S, 96, generator=torch.Generator().manual_seed(S)).cuda()
    ids = torch.randint(0, 5, (S, 1), generator=torch.Generator().manual_seed(S), dtype=torch.int32)
    _check(blocks, x, ids, "broadcast")
    few = ids.clone()
    few[:] = 2
    few[S // 2] = 4
    _check(blocks, x, few, "per_slot")


@pytest.mark.parametrize("S,n_in", [(129, 96), (200, 544), (255, 96), (256, 800), (257, 96)])
def test_slot_counts_over_many_experts(S, n_in):
    # up to 256 slots in one launch where the experts are many, however few of them are taken
    E, n_out = 60, 200
    blocks = _weights(E, n_out, n_in, S)
    g = torch.Generator().manual_seed(S)
    x = torch.randn(S, n_in, generator=g).to(torch.float16).cuda()
    ids = torch.randint(0, E, (S, 1), generator=g, dtype=torch.int32)
    _check(blocks, x, ids, "broadcast")
    ids[: S - 3] = torch.randint(57, 59, (S - 3, 1), generator=g, dtype=torch.int32)
    _check(blocks, x, ids, "per_slot")
    ids[5] = E
    ws = moe.workspace(S, 1, E, n_in, x_dtype=torch.float16)
    W = moe.weights_prepare(blocks.cuda(), E, n_out, n_in, wtype="mxfp4")
    moe.mul_mat_id_mx4(W, E, n_out, n_in, x, ids.cuda(), ws=ws)
    assert moe.get_status(ws) == moe.ERR_BAD_ID


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("stage", [0, 2])
def test_expired_wait_reports_timeout_and_the_device_recovers(T, stage):
    # one CTA's copy of one stage is never issued and the waits give up after a millisecond
    blocks = _weights(3, 300, 1600, 31)
    W = moe.weights_prepare(blocks.cuda(), 3, 300, 1600, wtype="mxfp4")
    x = torch.randn(T, 1600, generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
    ids = _ids(T, 2, 3, 32)
    ws = moe.workspace(T, 2, 3, 1600)
    moe.lib().moe_testing_stall(0, stage, 1000)
    try:
        moe.mul_mat_id_mx4(W, 3, 300, 1600, x, ids.cuda(), ws=ws)
        st = moe.get_status(ws)
    finally:
        moe.lib().moe_testing_stall(-1, 0, 0)
    assert st == moe.ERR_TIMEOUT
    site = int(ws[12:16].view(torch.int32).item())  # header word 3
    assert site >> 30 == 1 and 0 <= (site >> 20) & 0x3ff < 16
    torch.cuda.synchronize()
    assert moe.lib().moe_workspace_init(ws.data_ptr(), None) == moe.OK
    dst = moe.mul_mat_id_mx4(W, 3, 300, 1600, x, ids.cuda(), ws=ws)
    assert moe.get_status(ws) == moe.OK
    out, mag = ref.mx_product(blocks.numpy(), x.double().cpu().numpy(), ids.numpy(), False)
    assert (np.abs(dst.double().cpu().numpy() - out) <= 1600 * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("T", [4, 150])
def test_a_failed_call_leaves_later_ones_undone_until_the_status_is_read(T):
    blocks = _weights(4, 32, 64, 41)
    W = moe.weights_prepare(blocks.cuda(), 4, 32, 64, wtype="mxfp4")
    x = torch.randn(T, 64, generator=torch.Generator().manual_seed(1)).cuda()
    ids = _ids(T, 2, 4, 5).cuda()
    bad = ids.clone()
    bad[0, 0] = 4
    ws = moe.workspace(T, 2, 4, 64, x_dtype=torch.float32)
    out = torch.full((T, 2, 32), -7.0).cuda()
    moe.mul_mat_id_mx4(W, 4, 32, 64, x, bad, ws=ws, out=out)
    moe.mul_mat_id_mx4(W, 4, 32, 64, x, ids, ws=ws, out=out)
    assert moe.get_status(ws) == moe.ERR_BAD_ID
    assert (out == -7).all()
    moe.mul_mat_id_mx4(W, 4, 32, 64, x, ids, ws=ws, out=out)
    assert moe.get_status(ws) == moe.OK and not (out == -7).all()


def test_two_calls_at_once_on_two_streams():
    E, n_out, n_in, k = 8, 384, 1024, 2
    blocks = _weights(E, n_out, n_in, 43)
    W = moe.weights_prepare(blocks.cuda(), E, n_out, n_in, wtype="mxfp4")
    for T in (5, 400):
        xs = [torch.randn(T, n_in, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(2)]
        ids = [_ids(T, k, E, 50 + i).cuda() for i in range(2)]
        want = [moe.mul_mat_id_mx4(W, E, n_out, n_in, xs[i], ids[i]) for i in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        ws = [moe.workspace(T, k, E, n_in) for _ in range(2)]
        outs = [torch.empty(T, k, n_out).cuda() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(5):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    moe.mul_mat_id_mx4(W, E, n_out, n_in, xs[i], ids[i], ws=ws[i], out=outs[i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_many_calls_at_once_on_three_streams():
    # both forms, the general tables and the counted ones, with one another and with other kernels
    jobs = []
    for T, E, k, n_in, n_out in ((4, 64, 8, 512, 256), (300, 32, 4, 256, 300), (90, 1100, 4, 256, 64),
                                 (9000, 8, 4, 64, 128)):
        W = moe.weights_prepare(_weights(E, n_out, n_in, T).cuda(), E, n_out, n_in, wtype="mxfp4")
        g = torch.Generator().manual_seed(T)
        x = torch.randn(T, n_in, generator=g).bfloat16().cuda()
        ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
        args = (W, E, n_out, n_in, x, ids)
        jobs.append((args, moe.mul_mat_id_mx4(*args)))
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws = [[moe.workspace(a[5].shape[0], a[5].shape[1], a[1], a[3]) for a, _ in jobs] for _ in streams]
    outs = [[torch.empty_like(want) for _, want in jobs] for _ in streams]
    differ = [torch.zeros(1, dtype=torch.int64).cuda() for _ in streams]
    order = torch.randint(0, 12, (12000,), generator=torch.Generator().manual_seed(1)).tolist()
    torch.cuda.synchronize()
    for n, c in enumerate(order):
        i, j = c % 3, c // 3
        args, want = jobs[j]
        with torch.cuda.stream(streams[i]):
            moe.mul_mat_id_mx4(*args, ws=ws[i][j], out=outs[i][j])
            if n % 7 == 0:
                differ[i] += (outs[i][j] != want).any()
        if n % 60 == 59:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert [int(d.item()) for d in differ] == [0, 0, 0]
    assert all(moe.get_status(w) == moe.OK for row in ws for w in row)


def test_one_expert_takes_all_and_most_take_none():
    blocks = _weights(64, 64, 192, 1)
    x = torch.randn(600, 192, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    ids = torch.full((600, 1), 37, dtype=torch.int32)
    _check(blocks, x, ids, "broadcast")
    ids[::50] = 63
    _check(blocks, x, ids, "broadcast")


def test_the_same_expert_twice_in_a_token():
    blocks = _weights(4, 40, 64, 5)
    x = torch.randn(3, 64, generator=torch.Generator().manual_seed(6)).cuda()
    _check(blocks, x, torch.tensor([[1, 1], [0, 3], [2, 2]], dtype=torch.int32), "broadcast")


@pytest.mark.parametrize("T", [2, 70])
def test_wide_scales_and_zero_blocks(T):
    # block scales far apart in both operands, whole blocks of zeros, and a row of zeros
    g = torch.Generator().manual_seed(8)
    blocks = _weights(2, 96, 256, 9, 90, 160)
    blocks[:, ::3, 2, 1:] = 0
    x = torch.randn(T, 256, generator=g) * torch.exp2(torch.randint(-30, 30, (T, 8, 1), generator=g).float()
                                                      ).expand(T, 8, 32).reshape(T, 256)
    x[1] = 0
    x[0, 64:96] = 0
    _check(blocks, x.cuda(), _ids(T, 2, 2, 3), "broadcast")


@pytest.mark.parametrize("T", [2, 70])
def test_nan_rows_stay_in_their_rows(T):
    blocks = _weights(3, 50, 128, 11)
    x = torch.randn(T, 128, generator=torch.Generator().manual_seed(12)).cuda()
    x[1, 70] = float("nan")
    ids = _ids(T, 2, 3, 4)
    dst = _run(blocks, x, ids, "broadcast")
    assert torch.isnan(dst[1]).all()
    x[1] = 0
    clean = _run(blocks, x, ids, "broadcast")
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(dst[keep], clean[keep])


@pytest.mark.parametrize("T", [3, 80])
def test_bad_id_is_reported(T):
    blocks = _weights(4, 32, 64, 13)
    x = torch.randn(T, 64, generator=torch.Generator().manual_seed(1)).cuda()
    ids = _ids(T, 2, 4, 5)
    for bad in (-1, 4, 2 ** 30):
        b = ids.clone()
        b[T - 1, 1] = bad
        with pytest.raises(moe.MoeError) as e:
            _run(blocks, x, b, "broadcast")
        assert e.value.code == moe.ERR_BAD_ID
    _check(blocks, x, ids, "broadcast")


@pytest.mark.parametrize("T", [4, 200])
def test_results_follow_the_rounded_values(T):
    # the product of the rounded operands: mul_mat_id on the values that the quantiser returns
    E, n_out, n_in, k = 8, 144, 320, 3
    blocks = _weights(E, n_out, n_in, 15)
    x = torch.randn(T, n_in, generator=torch.Generator().manual_seed(16)).bfloat16().cuda()
    ids = _ids(T, k, E, 17)
    dst = _run(blocks, x, ids, "broadcast")
    _, values = moe.mxfp4_quantize(x, with_values=True)
    W = moe.weights_prepare(blocks.cuda(), E, n_out, n_in, wtype="mxfp4")
    other = moe.mul_mat_id(W, E, n_out, n_in, values, ids.cuda(), wtype="mxfp4")
    _, mag = ref.mx_product(blocks.numpy(), x.double().cpu().numpy(), ids.numpy(), False)
    assert (np.abs((dst - other).double().cpu().numpy()) <= 2 * n_in * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("T", [4, 100])
def test_graph_replay_rows_behind_and_two_workspaces(T):
    E, n_out, n_in, k = 8, 100, 224, 2
    blocks = _weights(E, n_out, n_in, 19)
    W = moe.weights_prepare(blocks.cuda(), E, n_out, n_in, wtype="mxfp4")
    g = torch.Generator().manual_seed(20)
    x = torch.randn(T, n_in, generator=g).bfloat16().cuda()
    ids = _ids(T, k, E, 21).cuda()
    ws = moe.workspace(T, k, E, n_in)
    out = torch.full((T + 2, k, n_out), -7.0).cuda()
    moe.mul_mat_id_mx4(W, E, n_out, n_in, x, ids, ws=ws, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.mul_mat_id_mx4(W, E, n_out, n_in, x, ids, ws=ws, out=out)
    x2 = torch.randn(T, n_in, generator=g).bfloat16().cuda()
    ids2 = _ids(T, k, E, 22).cuda()
    x.copy_(x2)
    ids.copy_(ids2)
    for _ in range(3):
        graph.replay()
    assert moe.get_status(ws) == moe.OK
    assert (out[T:] == -7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws2 = moe.workspace(T, k, E, n_in)
        other = moe.mul_mat_id_mx4(W, E, n_out, n_in, x2, ids2, ws=ws2)
    side.synchronize()
    assert torch.equal(out[:T], other)


def test_no_tokens():
    blocks = _weights(4, 32, 64, 23)
    assert _run(blocks, torch.empty(0, 64).cuda(), torch.empty(0, 2, dtype=torch.int32), "broadcast").shape == (0, 2, 32)


@pytest.mark.parametrize("T", [3, 90])
def test_layer_forward_and_router_gradient(T):
    # route_scored -> product of quantised experts -> combine, and back to the logits
    E, n_in, n_out, k = 16, 128, 96, 4
    g = torch.Generator().manual_seed(T)
    blocks = moe.mxfp4_quantize(torch.randn(E, n_out, n_in, generator=g).cuda())
    W = moe.weights_prepare(blocks, E, n_out, n_in, wtype="mxfp4")
    x = torch.randn(T, n_in, generator=g).bfloat16().cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    bias = (torch.randn(E, generator=g) * 0.05).cuda()
    kw = dict(score="sigmoid", normalize=True, scale=2.5)
    ids, w = moe.route_scored(logits, k, bias=bias, n_groups=4, topk_groups=2, group_score="top2", **kw)
    dst = moe.mul_mat_id_mx4(W, E, n_out, n_in, x, ids)
    y = moe.combine(dst, w)
    dy = torch.randn(T, n_out, generator=g).cuda()
    dw, ddst = moe.combine_backward(dy, dst, w)
    dl = moe.route_scored_backward(logits, ids, dw, **kw)
    # the 64-bit layer on the same choice
    l = logits.double().cpu().numpy()
    r_ids, r_w, _ = ref.route(l, k, bias.double().cpu().numpy(), "sigmoid", 4, 2, "top2", True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    r_dst, mag = ref.mx_product(blocks.cpu().numpy(), x.double().cpu().numpy(), r_ids, False)
    r_y = np.einsum("tk,tkn->tn", r_w, r_dst)
    r_dw, _, r_dd = ref.combine_grad(dy.cpu().numpy(), r_dst, r_w)
    r_dl, _ = ref.route_grad(l, r_ids, r_dw, "sigmoid", True, 2.5, ref.U)
    # every stage's bound is below 2^-15 of the magnitudes it sums
    rel = 2.0 ** -15
    assert (np.abs(y.double().cpu().numpy() - r_y) <= rel * np.einsum("tk,tkn->tn", r_w, mag)).all()
    mag_dw = np.einsum("tn,tkn->tk", np.abs(dy.double().cpu().numpy()), mag)
    assert (np.abs(dw.double().cpu().numpy() - r_dw) <= rel * mag_dw).all()
    assert (np.abs(ddst.double().cpu().numpy() - r_dd) <= rel * np.abs(r_dd) + 1e-30).all()
    assert (np.abs(dl.double().cpu().numpy() - r_dl) <= rel * 2.5 * 2 * mag_dw.max(1, keepdims=True)).all()
