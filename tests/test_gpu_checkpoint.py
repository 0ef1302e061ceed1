"""8-bit rows: codes and scales bit for bit, and back."""
import math

import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import products as op
from product_util import Guarded, normal

pytestmark = pytest.mark.gpu

MX, ROW = fq.FQ_F8_MX, fq.FQ_F8_ROW


def values(rows, cols, seed=0):
    """Values of very different magnitudes, zeros and subnormals among them."""
    x = normal(seed, rows, cols, dtype=torch.float32) * torch.exp(4 * normal(seed + 1, rows, 1, dtype=torch.float32))
    x = x * torch.exp(normal(seed + 2, rows, cols, dtype=torch.float32))
    x[:, ::7] = 0
    if rows > 3:
        x[1] = 0
        x[2] *= 1e-38
        x[3] *= 1e30
    return x.to(torch.bfloat16)


def encode(x, f8):
    rows, cols = x.shape
    g = Guarded()
    codes = g.output((rows, cols), torch.uint8)
    scales = g.output((rows, cols // 32), torch.uint8) if f8 == MX else g.output((rows,), torch.float32)
    fq.fq_f8_encode(g.input(x), f8, codes=codes, scales=scales)
    y = g.output((rows, cols), torch.bfloat16)
    fq.fq_f8_decode(codes, scales, f8, y=y)
    torch.cuda.synchronize()
    g.check()
    return codes, scales, y


def check(x, f8):
    codes, scales, y = encode(x, f8)
    want, want_scales = op.encode_mx(x) if f8 == MX else op.encode_row(x)
    nan = torch.isnan(want_scales) if f8 == ROW else torch.zeros_like(want_scales, dtype=torch.bool)
    assert torch.equal(scales[~nan], want_scales[~nan]) and bool(torch.isnan(scales[nan]).all() if f8 == ROW else True)
    assert torch.equal(codes, want)
    back = op.decode(codes, scales, f8 == MX).float().to(torch.bfloat16)
    fine = ~torch.isnan(back)
    assert torch.equal(y[fine], back[fine]) and bool(torch.isnan(y[~fine]).all())


COLS = [32, 64, 96, 128, 160, 512, 544, 1024, 2048, 2080, 2880, 4096, 4128, 8192, 8224, 32768]


@pytest.mark.parametrize("f8", [MX, ROW])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 5, 67])
def test_encode_decode(f8, cols, rows):
    check(values(rows, cols, rows + cols), f8)


@pytest.mark.parametrize("f8", [MX, ROW])
def test_large(f8):
    check(values(4099, 2880), f8)


def test_wide_rows_in_blocks():
    check(values(3, 65568), MX)
    x = values(3, 40000)
    codes = torch.zeros((3, 40000), dtype=torch.uint8, device=DEV)
    y = fq.fq_f8_decode(codes, torch.ones(3, device=DEV), ROW)
    assert not bool(y.any())
    with pytest.raises(fq.FqError) as e:
        fq.fq_f8_encode(x, ROW)
    assert e.value.status == fq.FQ_ERR_SHAPE


@pytest.mark.parametrize("f8", [MX, ROW])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_not_finite(f8, bad):
    x = values(6, 96)
    x[4, 40] = bad
    check(x, f8)


@pytest.mark.parametrize("f8", [MX, ROW])
def test_every_bf16(f8):
    """Every finite BF16 value, alone in a block of zeros and beside its neighbours."""
    bits = torch.arange(1 << 16, dtype=torch.int32, device=DEV).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = torch.where(torch.isfinite(v), v, torch.zeros((), dtype=torch.bfloat16, device=DEV))
    check(v.view(-1, 64), f8)
    x = torch.zeros((1 << 16, 32), dtype=torch.bfloat16, device=DEV)
    x[:, 5] = v
    check(x, f8)


def test_same_as_the_norm_writes():
    """fq_rmsnorm_fwd's 8-bit output is the encoding of what its BF16 output is
    rounded from: where that is exact the two agree."""
    x = torch.ones((9, 64), dtype=torch.bfloat16, device=DEV)
    gamma = torch.pow(2.0, torch.arange(64, device=DEV).float() % 9 - 4)
    _, y = fq.fq_rmsnorm_fwd(x, gamma, 0.0)
    for f8 in (MX, ROW):
        _, codes, scales = fq.fq_rmsnorm_fwd(x, gamma, 0.0, f8=f8)
        again = fq.fq_f8_encode(y, f8)
        assert torch.equal(codes, again[0]) and torch.equal(scales, again[1])
