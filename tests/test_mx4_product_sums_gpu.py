"""The 4-bit product's sums.  Where every partial sum is a multiple of one unit and
below 2^24 of them, float32 holds it exactly, in whatever order it is formed:
results have to equal the 64-bit ones bit for bit, so that a block with another
block's scale, or a row of another plane, cannot hide in a tolerance.  Where
scales lie far apart the bound is that of a float sum by instructions: the 32
products of a block are integers over one power of two and their sum is exact
(at most 32 * 144 units), and an instruction adds two such blocks to the sum so far,
each of the three cut, and the result rounded, by less than a unit of the last
place of the largest: 4 * 2^-23 of the terms' magnitudes for 64 values, n_in / 8 * 2^-24
in all."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_b200 as moe
from tests import routed_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _weights(E, n_out, n_in, seed, lo, hi):
    g = torch.Generator().manual_seed(seed)
    b = torch.randint(0, 256, (E, n_out, n_in // 32, 17), generator=g, dtype=torch.uint8)
    b[..., 0] = torch.randint(lo, hi, (E, n_out, n_in // 32), generator=g, dtype=torch.uint8)
    return b


def _rows(rows, n_in, seed, spread=3):
    """Normal values, blocks of 32 scaled by 1, 2, 4 (spread 3)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n_in, generator=g)
    s = torch.exp2(torch.randint(0, spread, (rows, n_in // 32, 1), generator=g).float())
    return (x.view(rows, -1, 32) * s).view(rows, n_in)


def _ids(T, k, E, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()


def _run(blocks, x, ids, mode):
    E, n_out, nb, _ = blocks.shape
    W = moe.weights_prepare(blocks.cuda(), E, n_out, nb * 32, wtype="mxfp4")
    return moe.mul_mat_id_mx4(W, E, n_out, nb * 32, x, ids.cuda(), mode=mode)


def _exactly(blocks, x, ids, mode):
    dst = _run(blocks, x, ids, mode).double().cpu().numpy()
    out, mag = ref.mx_product(blocks.numpy(), x.double().cpu().numpy(), ids.numpy(), mode == "per_slot")
    # the unit: half times half under the smallest scales
    unit = 0.25 * 2.0 ** (int(blocks[..., 0].min()) - 127.0 + int(ref.mx_round(x.double().cpu().numpy())[1].min()) - 127.0)
    assert (mag / unit).max() < 2 ** 24
    assert np.array_equal(dst, out), np.argwhere(dst != out)[:4].tolist()


# the one-launch form up to 36 planes of 256 values, then the GEMM; rows of more than 32 groups of four planes
@pytest.mark.parametrize("T,n_in", [(2, 7168), (2, 9216), (2, 9248), (1, 12320), (120, 9216), (120, 9248), (3, 32768),
                                    (3, 32800), (70, 33024)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_rows_exactly(T, n_in, dtype):
    blocks = _weights(2, 20, n_in, n_in, 120, 123)
    _exactly(blocks, _rows(T, n_in, T).to(DT[dtype]).cuda(), _ids(T, 2, 2, 1), "broadcast")


@pytest.mark.parametrize("mode", ["broadcast", "per_slot"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,k,n_in", [(40, 7, 1056), (90, 3, 1312), (33, 9, 64)])
def test_more_than_1024_experts_exactly(mode, dtype, T, k, n_in):
    # tables by the general row-id pass, rows rounded by a launch of their own
    blocks = _weights(1100, 17, n_in, k, 120, 123)
    x = _rows(T if mode == "broadcast" else T * k, n_in, T).to(DT[dtype]).cuda()
    _exactly(blocks, x, _ids(T, k, 1100, T), mode)


@pytest.mark.parametrize("mode", ["broadcast", "per_slot"])
@pytest.mark.parametrize("T,E,k,n_in,n_out", [(4, 64, 8, 2048, 130), (64, 30, 4, 1440, 300), (500, 12, 3, 2880, 272)])
def test_usual_rows_exactly(mode, T, E, k, n_in, n_out):
    blocks = _weights(E, n_out, n_in, E, 120, 123)
    x = _rows(T if mode == "broadcast" else T * k, n_in, T).bfloat16().cuda()
    _exactly(blocks, x, _ids(T, k, E, T), mode)


# every row at one magnitude, from the smallest of the type to the largest
@pytest.mark.parametrize("T", [12, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_of_extreme_magnitudes(T, dtype):
    n_in, n_out = 160, 40
    info = torch.finfo(DT[dtype])
    low, high = np.log2(info.tiny), np.log2(info.max)
    exps = torch.cat([low - 6 + torch.arange(T // 2) % 12, high - 1 - torch.arange(T - T // 2) % 12])
    g = torch.Generator().manual_seed(T)
    v = torch.rand(T, n_in, generator=g).double() + 1
    v[torch.rand(T, n_in, generator=g) < 0.5] *= -1
    x = (v * torch.exp2(torch.floor(exps.double()))[:, None]).clamp(info.min, info.max).to(DT[dtype])
    x[1, :64] = 0
    x[2, 32:] = 0
    x[T - 1] = info.max
    # an expert for the small rows, one for the large ones: results near 1
    blocks = _weights(2, n_out, n_in, 5, 120, 123)
    blocks[0, ..., 0] += 90 if dtype != "f16" else 10
    blocks[1, ..., 0] -= 90 if dtype != "f16" else 10
    ids = (torch.arange(T) >= T // 2).int()[:, None]
    dst = _run(blocks, x.cuda(), ids, "broadcast").double().cpu().numpy()
    out, _ = ref.mx_product(blocks.numpy(), x.double().numpy(), ids.numpy(), False)
    # a row's scales are at most 4 apart and the weights' 4: 160 * 144 * 16 units fit 24 bits
    assert np.array_equal(dst, out), np.argwhere(dst != out)[:4].tolist()
    _, values = moe.mxfp4_quantize(x.cuda(), with_values=True)
    assert np.array_equal(dst, _run(blocks, values, ids, "broadcast").double().cpu().numpy())


@pytest.mark.parametrize("T,E,k,n_in,n_out", [(2, 4, 2, 7168, 200), (150, 4, 2, 7168, 200), (300, 3, 2, 2880, 144)])
def test_scales_far_apart(T, E, k, n_in, n_out):
    # blocks of both operands spread over 2^24 and 2^20
    blocks = _weights(E, n_out, n_in, 9, 108, 133)
    x = _rows(T, n_in, T, spread=21).cuda()
    ids = _ids(T, k, E, T)
    dst = _run(blocks, x, ids, "broadcast").double().cpu().numpy()
    out, mag = ref.mx_product(blocks.numpy(), x.double().cpu().numpy(), ids.numpy(), False)
    ratio = np.abs(dst - out) / (n_in / 8 * 2.0 ** -24 * mag)
    print("largest share of the bound: %.3f" % ratio.max())
    assert (ratio <= 1).all(), float(ratio.max())
