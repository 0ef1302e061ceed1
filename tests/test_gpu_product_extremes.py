"""The feed-forward products' backward where its values come near the ends of their
types' ranges."""
import math

import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import products as op
from product_util import normal, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 150])
@pytest.mark.parametrize("size", [1e-3, 1.0])
@pytest.mark.parametrize("gate", [False, True])
def test_largest_gradients_with_a_scale_per_row(rows, size, gate):
    """dz is finite in BF16, but not times a mantissa from 1 to 2: dw stays what the
    formula says, 0 where x is 0 among it.  One row has the large gradients, so that
    dw is a single product and no sum of several overflows: |x| below 1.5 times 2.5e38
    below FP32's largest."""
    k, n = 64, 32
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device=DEV)
    # every other column is 0; the largest is 448 * 1.75 / 1024 times `size`: a scale of mantissa 1.75
    x[:, ::2] = (normal(0, rows, k // 2, dtype=torch.float32).clamp(-2, 2) / 4 * size).to(torch.bfloat16)
    x[:, 0] = 448 * 1.75 / 1024 * size
    codes, scales = op.encode_row(x)
    dy = torch.zeros((rows, n), dtype=torch.bfloat16, device=DEV)
    dy[rows // 2] = 2.5e38
    dy[rows // 2, ::3] = -2.5e38
    pre = torch.ones((rows, 2 * n if gate else n), dtype=torch.bfloat16, device=DEV)
    w = normal(1, k, 2 * n if gate else n, sigma=1e-6)
    kw = dict(act=op.RELU, x_f8=fq.FQ_F8_ROW, x_scales=scales, dw_dtype=torch.float32, need_dx=False, need_dbias=False)
    xv = op.decode(codes, scales, False)
    if gate:
        _, dw, _ = fq.fq_glu_bwd(dy, codes, w, pre, **kw)
        v, t = op.glu_bwd(dy, xv, w, pre, (op.RELU, 1.0, math.inf, 0.0), dw_dtype=torch.float32)
    else:
        _, dw, _ = fq.fq_linear_bwd(dy, codes, w, pre=pre, **kw)
        v, t = op.linear_bwd(dy, xv, w, pre, op.RELU, dw_dtype=torch.float32)
    assert bool((scales.frexp().mantissa > 0.51).all()) and float(xv.abs().max()) < 1.5
    within(dw, v["dw"], t["dw"], "dw")
    assert bool((dw[1::2] == 0).all())


@pytest.mark.parametrize("top", [2.0 ** 106, 2.0 ** 109, 3.3e38])
def test_largest_activations_with_a_scale_per_row(top):
    """Scales on both sides of 2^100 (448 times which is 2^108.8) and the largest there are."""
    rows, k, n = 70, 64, 32
    x = (normal(0, rows, k, dtype=torch.float32).clamp(-3, 3) / 3 * top).to(torch.bfloat16)
    x[:, 0] = top
    codes, scales = op.encode_row(x)
    dy, pre = normal(1, rows, n, sigma=1e-4), torch.ones((rows, n), dtype=torch.bfloat16, device=DEV)
    _, dw, _ = fq.fq_linear_bwd(dy, codes, normal(2, k, n), pre=pre, act=op.RELU, x_f8=fq.FQ_F8_ROW, x_scales=scales,
                                dw_dtype=torch.float32, need_dx=False, need_dbias=False)
    v, t = op.linear_bwd(dy, op.decode(codes, scales, False), normal(2, k, n), pre, op.RELU, dw_dtype=torch.float32)
    within(dw, v["dw"], t["dw"], "dw")


def test_rows_that_stand_for_nan():
    """An infinite activation makes its row NaN in 8 bits: so is dw, and dx is not."""
    rows, k, n = 70, 64, 32
    x = normal(0, rows, k)
    x[3, 5] = math.inf
    codes, scales = op.encode_row(x)
    dx, dw, _ = fq.fq_linear_bwd(normal(1, rows, n), codes, normal(2, k, n), pre=normal(3, rows, n), act=op.SILU,
                                 x_f8=fq.FQ_F8_ROW, x_scales=scales)
    assert bool(dw.isnan().all()) and bool(dx.isfinite().all())


@pytest.mark.parametrize("dh,u,g", [(2.5e38, 4.0, -9.0), (-2.5e38, 100.0, -12.0), (1e3, 1e36, -200.0), (3e-3, 3.3e38, 2.4), (2e-38, 1e6, -9.0)])
@pytest.mark.parametrize("kind", [op.SILU, op.GELU])
def test_gate_of_large_values(dh, u, g, kind):
    """dh (u + shift) a'(g) is finite, dh (u + shift) may not be: dg from the bias gradient
    of one row, to 2^-24 of three products and the slope's own bound."""
    n = 32
    h = torch.full((1, n), dh, dtype=torch.bfloat16, device=DEV)
    pre = torch.cat([torch.full((1, n), v, dtype=torch.bfloat16, device=DEV) for v in (g, u)], 1)
    x, w = torch.zeros((1, 8), dtype=torch.bfloat16, device=DEV), torch.zeros((8, 2 * n), dtype=torch.bfloat16, device=DEV)
    _, _, dbias = fq.fq_glu_bwd(h, x, w, pre, act=kind, need_dx=False, need_dw=False)
    value, slope, tv, td = op.act_close(pre[0, :n], kind)
    up, d = pre[0, n:].double(), h[0].double()
    for got, want, bound in ((dbias[:n], d * slope * up, td * (d * up).abs()), (dbias[n:], d * value, tv * d.abs())):
        within(got, want, bound + 3 * op.EPS32 * want.abs() + 2.0 ** -140, "dbias")
