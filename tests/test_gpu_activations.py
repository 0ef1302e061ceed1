"""SiLU and GELU of the feed-forward products over their whole range, relative to their
values (oracle.products.act_close): the forward through an FP32 output of a product that
is nothing but its bias, the slope through the FP32 bias gradient of a single row."""
import math

import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import products as op
from product_util import within

pytestmark = pytest.mark.gpu

ACTS = {"silu": (op.SILU, 90.0), "gelu": (op.GELU, 14.0)}


def all_bf16(top):
    """Every BF16 value of at most `top` in magnitude, and zeros up to a multiple of eight."""
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    v = v[v.abs() <= top]
    return torch.cat((v, torch.zeros(-v.numel() % 8))).to(DEV)


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("rows", [1, 70])
def test_value(name, rows):
    kind, top = ACTS[name]
    z = torch.cat((torch.linspace(-top, top, 1 << 16, device=DEV), all_bf16(top)))
    n = z.numel()
    y = torch.empty((rows, n), device=DEV)
    fq.fq_linear_fwd(torch.zeros((rows, 8), dtype=torch.bfloat16, device=DEV), torch.zeros((8, n), dtype=torch.bfloat16, device=DEV),
                     bias=z, act=kind, y=y)
    value, _, bound, _ = op.act_close(z, kind)
    within(y, value.expand(rows, n), bound.expand(rows, n), name)


@pytest.mark.parametrize("name", list(ACTS))
def test_slope(name):
    kind, top = ACTS[name]
    z = all_bf16(top)
    n = z.numel()
    one = torch.ones((1, n), dtype=torch.bfloat16, device=DEV)
    x, w = torch.zeros((1, 8), dtype=torch.bfloat16, device=DEV), torch.zeros((8, n), dtype=torch.bfloat16, device=DEV)
    _, _, dbias = fq.fq_linear_bwd(one, x, w, pre=z.to(torch.bfloat16)[None], act=kind, need_dx=False, need_dw=False)
    _, slope, _, bound = op.act_close(z, kind)
    within(dbias, slope, bound, name)


@pytest.mark.parametrize("name,alpha", [("silu", 1.0), ("silu", 1.702), ("gelu", 1.0)])
def test_gate(name, alpha):
    """With u = 1 and dh = 1 the gate's bias gradient is a'(g), the other half's a(g)."""
    kind, top = ACTS[name]
    z = all_bf16(top / alpha)
    n = z.numel()
    one = torch.ones((1, n), dtype=torch.bfloat16, device=DEV)
    x, w = torch.zeros((1, 8), dtype=torch.bfloat16, device=DEV), torch.zeros((8, 2 * n), dtype=torch.bfloat16, device=DEV)
    _, _, dbias = fq.fq_glu_bwd(one, x, w, torch.cat((z.to(torch.bfloat16)[None], one), 1), act=kind, alpha=alpha, limit=math.inf,
                                need_dx=False, need_dw=False)
    value, slope, tv, td = op.act_close(z, kind, float(torch.tensor(alpha, dtype=torch.float32)))
    within(dbias[:n], slope, td, name + "'s slope")
    within(dbias[n:], value, tv, name)
