"""moe_mxfp4_quantize against a 64-bit implementation, bit for bit: every
midpoint and neighbour of the E2M1 grid, scales from the smallest to the
largest, subnormals, zeros, NaN and infinities, strided rows, odd counts; and
the blocks it makes through weight preparation and the existing product."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_b200 as moe
from tests import routed_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _check(x):
    blocks, values = moe.mxfp4_quantize(x, with_values=True)
    v, X, code = ref.mx_round(x.double().cpu().numpy())
    assert np.array_equal(blocks.cpu().numpy(), ref.mx_blocks(X, code))
    assert values.dtype == x.dtype
    assert np.array_equal(values.double().cpu().numpy(), v, equal_nan=True)
    assert torch.equal(moe.mxfp4_quantize(x), blocks)
    return blocks, values


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (5, 7168), (65, 96), (2, 3, 128), (1000, 2880), (32,)])
def test_quantize(dtype, shape):
    g = torch.Generator().manual_seed(shape[-1])
    x = torch.randn(*shape, generator=g) * torch.exp2(torch.randn(*shape[:-1], 1, generator=g) * 4)
    _check(x.to(DT[dtype]).cuda())


def test_every_border_of_the_grid():
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0, 0.5, 1, 1.5, 2, 3, 4, 6, 7.9], np.float32)
    cand = np.concatenate([mid, np.nextafter(mid, np.float32(9)), np.nextafter(mid, np.float32(-9))])
    cand = np.concatenate([cand, -cand])
    rows = []
    for ex in (-126, -30, 0, 1, 90):
        for top in (4.0, 6.0, 7.75):
            for i in range(0, len(cand), 31):
                r = np.zeros(32, np.float32)
                c = cand[i:i + 31]
                r[:len(c)] = c
                r[31] = top
                rows.append(np.ldexp(r, ex))
    _check(torch.from_numpy(np.stack(rows)).cuda())


def test_extreme_magnitudes():
    f = np.float32
    vals = [np.ldexp(f(1), e) for e in (-149, -140, -127, -126, -125, -124, -123, -60, 0, 60, 126, 127)]
    vals += [np.finfo(f).max, f(0)]
    rows = np.zeros((len(vals), 32), f)
    for i, v in enumerate(vals):
        rows[i] = v * np.linspace(-1, 1, 32).astype(f)
        rows[i, 5] = v
        rows[i, 6] = -0.0
    x = torch.from_numpy(rows).cuda()
    _check(x)
    _check(x.bfloat16())
    h = torch.tensor([2.0 ** -24, 2.0 ** -23, 2.0 ** -14, 1.0, 65504.0])[:, None] * torch.linspace(-1, 1, 64)
    _check(h.half().cuda())


def test_nan_and_infinity_mark_their_block_only():
    x = torch.randn(4, 96, generator=torch.Generator().manual_seed(1))
    x[0, 3] = float("nan")
    x[1, 40] = float("inf")
    x[2, 95] = -float("inf")
    for d in DT.values():
        blocks, values = _check(x.to(d).cuda())
        assert torch.isnan(values).sum().item() == 3 * 32
        assert (blocks[..., 0] == 255).sum().item() == 3


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad", [1, 8, 32])
def test_strided_and_misaligned_rows(dtype, pad):
    g = torch.Generator().manual_seed(pad)
    wide = torch.randn(9, 160 + pad, generator=g).to(DT[dtype]).cuda()
    _check(wide[:, :160])
    _check(wide[:, pad:])
    out = torch.full((9 * 5 * 17 + 64,), 77, dtype=torch.uint8).cuda()
    moe.mxfp4_quantize(wide[:, :160], out=out[3:])
    ref_blocks = moe.mxfp4_quantize(wide[:, :160].contiguous())
    assert torch.equal(out[3:3 + 9 * 5 * 17], ref_blocks.reshape(-1))
    assert (out[:3] == 77).all() and (out[3 + 9 * 5 * 17:] == 77).all()


def test_blocks_feed_the_weight_preparation():
    E, n_out, n_in, T, k = 4, 48, 96, 5, 2
    g = torch.Generator().manual_seed(3)
    w = torch.randn(E, n_out, n_in, generator=g).cuda()
    blocks, values = moe.mxfp4_quantize(w, with_values=True)
    W = moe.weights_prepare(blocks, E, n_out, n_in, wtype="mxfp4")
    x = torch.randn(T, n_in, generator=g).bfloat16().cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    dst = moe.mul_mat_id(W, E, n_out, n_in, x, ids, wtype="mxfp4").double()
    exact = torch.einsum("tkon,tn->tko", values.double()[ids.long()], x.double())
    mag = torch.einsum("tkon,tn->tko", values.double().abs()[ids.long()], x.double().abs())
    assert ((dst - exact).abs() <= 2e-3 * mag + 1e-5).all()


def test_empty():
    assert moe.mxfp4_quantize(torch.empty(0, 64).cuda()).shape == (0, 2, 17)
