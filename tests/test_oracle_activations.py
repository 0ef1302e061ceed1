"""The oracle's close bounds of SiLU and GELU: they hold for an FP32 evaluation of the
formulas, and tell a side that is cut to 0 from one that is computed."""
import math

import pytest
import torch

from oracle import products as op


def sweep(kind, alpha=1.0):
    top = 13.0 if kind == op.GELU else 86.0 / alpha
    return torch.linspace(-top, top, 20001, dtype=torch.float32)


@pytest.mark.parametrize("kind,alpha", [(op.SILU, 1.0), (op.SILU, 1.702), (op.GELU, 1.0)])
def test_values(kind, alpha):
    """Where the usual formulas do not cancel they are the same."""
    z = sweep(kind, alpha).double()
    v, d = op.act(z, kind, alpha)
    value, slope, _, _ = op.act_close(z, kind, alpha)
    assert torch.allclose(v, value, rtol=1e-12, atol=1e-14) and torch.allclose(d, slope, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("kind,alpha", [(op.SILU, 1.0), (op.SILU, 1.702), (op.GELU, 1.0)])
def test_differences(kind, alpha):
    """The slope against differences of the value, relative to the value on the far side.
    Central differences are off by step^2 / 6 times the third derivative, which is below
    (|z| + |alpha| + 3)^3 times value and slope there."""
    z = sweep(kind, alpha).double()
    step = 1e-5
    _, slope, _, _ = op.act_close(z, kind, alpha)
    value = [op.act_close(z + s * step, kind, alpha)[0] for s in (-1, 0, 1)]
    size = (z.abs() + abs(alpha) + 3) ** 3 * (value[1].abs() + slope.abs()).clamp_min(1e-300)
    assert bool(((value[2] - value[0]) / (2 * step) - slope).abs().le(size * step ** 2 + value[1].abs() * 1e-15 * 4 / step).all())


@pytest.mark.parametrize("kind,alpha", [(op.SILU, 1.0), (op.SILU, 1.702), (op.GELU, 1.0)])
def test_far_side_is_told_from_zero(kind, alpha):
    """A planted 0 is refused wherever the value is not there, a planted constant slope
    wherever the slope is not: the bounds are a thousandth of them at most."""
    z = sweep(kind, alpha)
    value, slope, tv, td = op.act_close(z, kind, alpha)
    assert bool((tv[z != 0] < 1e-3 * value[z != 0].abs()).all())
    # a' crosses 0 at -1.2785 / alpha and -0.7518
    away = (z.double() + (1.2785 / alpha if kind == op.SILU else 0.7518)).abs() > 0.05
    assert bool((td[away] < 1e-3 * slope[away].abs()).all())


@pytest.mark.parametrize("alpha", [1.0, 1.702])
def test_silu_in_fp32(alpha):
    """The formulas step by step in FP32, each step rounded once."""
    z = sweep(op.SILU, alpha)
    a = torch.tensor(alpha, dtype=torch.float32)
    v = a * z
    e = torch.exp2((v * torch.tensor(-math.log2(math.e), dtype=torch.float32)).double()).float()
    s = (1 / (1 + e).double()).float()
    value, slope, tv, td = op.act_close(z, op.SILU, float(a))
    got = z * s
    assert bool(((got.double() - value).abs() <= tv).all())
    got = (a.double() * (got * (1 - s)).double() + s.double()).float()
    assert bool(((got.double() - slope).abs() <= td).all())
