"""The oracle of the feed-forward products against differences and against
torch's own functions."""
import math

import pytest
import torch

from oracle import products as op

GATES = {"silu": (op.SILU, 1.0, math.inf, 0.0), "gelu": (op.GELU, 1.0, math.inf, 0.0),
         "clamped": (op.SILU, 1.702, 1.25, 1.0), "relu": (op.RELU, 1.0, math.inf, 0.0)}


def normal(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("kind", [op.NONE, op.RELU, op.SILU, op.GELU])
def test_activations(kind):
    z = normal(1000) * 3
    fn = {op.NONE: lambda v: v, op.RELU: torch.relu, op.SILU: torch.nn.functional.silu, op.GELU: torch.nn.functional.gelu}[kind]
    v, d = op.act(z, kind)
    assert torch.allclose(v, fn(z), atol=1e-14)
    step = 1e-5
    # central differences are off by step^2 / 6 times the third derivative (below 2)
    assert torch.allclose(d, (fn(z + step) - fn(z - step)) / (2 * step), atol=1e-9) or kind == op.RELU
    assert kind != op.RELU or torch.equal(d, (z > 0).double())


@pytest.mark.parametrize("name", list(GATES))
@pytest.mark.parametrize("starts", [None, [0, 3, 3, 7]])
def test_glu_gradients(name, starts):
    """Against autograd of the forward, and against differences of it."""
    g = GATES[name]
    rows, k, n = 8 if starts else 7, 5, 6
    x, w, dh = normal(rows, k, seed=1), normal(*([3] if starts else []), k, 2 * n, seed=2), normal(rows, n, seed=3)
    end = starts[-1] if starts else rows

    def loss(x, w):
        return (op.glu_fwd(x, w, None, g, starts)[0]["y"][:end] * dh[:end]).sum()

    pre = op.glu_fwd(x, w, None, g, starts)[0]["z"]
    v, _ = op.glu_bwd(dh, x, w, pre, g, starts)
    step = 1e-6
    for at in ((0, 0), (2, 4), (end - 1, 1)):
        e = torch.zeros_like(x)
        e[at] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - v["dx"][at]) < 1e-7
    for at in ((0, 0), (4, 2 * n - 1), (2, n)):
        at = (0,) + at if starts else at
        e = torch.zeros_like(w)
        e[at] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - v["dw"][at]) < 1e-7
    if starts:
        assert not v["dw"][1].any() and not v["dbias"][1].any()


@pytest.mark.parametrize("kind", [op.NONE, op.SILU, op.GELU])
def test_linear_gradients(kind):
    x, w, b, dy = normal(6, 4, seed=1).requires_grad_(), normal(4, 5, seed=2).requires_grad_(), normal(5, seed=3).requires_grad_(), normal(6, 5, seed=4)
    fn = {op.NONE: lambda v: v, op.SILU: torch.nn.functional.silu, op.GELU: torch.nn.functional.gelu}[kind]
    z = x @ w + b
    fn(z).backward(dy)
    v, _ = op.linear_bwd(dy, x.detach(), w.detach(), z.detach(), kind)
    for got, want in ((v["dx"], x.grad), (v["dw"], w.grad), (v["dbias"], b.grad)):
        assert torch.allclose(got, want, atol=1e-12)


def test_e4m3():
    v = op.e4m3_values()
    assert torch.equal(v.float(), torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float())
    a = torch.cat((v, (v[1:] + v[:-1]) / 2, (v[1:] * 0.51 + v[:-1] * 0.49)))
    a = torch.cat((a, -a))
    assert torch.equal(op._nearest(a).to(torch.uint8), a.float().to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("mx", [True, False])
def test_encode_decode(mx):
    x = (normal(9, 96) * torch.exp(normal(9, 96, seed=1))).to(torch.bfloat16)
    x[3] = 0
    codes, scales = (op.encode_mx if mx else op.encode_row)(x)
    back = op.decode(codes, scales, mx)
    # half a step of E4M3, or of its subnormals under the scale
    s = op.pow2(scales.long() - 127).repeat_interleave(32, 1) if mx else scales.double()[:, None]
    assert ((back - x.double()).abs() <= 2.0 ** -4 * x.double().abs() * (1 + 2.0 ** -20) + 2.0 ** -10 * s).all()
    assert (back.abs() <= 448 * s).all()
