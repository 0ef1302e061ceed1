"""The training step that runs the row operators together with the quantized
linears: its gradients against torch's autograd of the same block in FP32, and a
few steps of it."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_step  # noqa: E402

pytestmark = pytest.mark.gpu


def test_gradients_with_plain_products():
    """With plain products what differs from autograd in FP32 is the 8-bit rounding
    of the experts' and the router's input, at most 2^-4 and in the mean of squares
    about 2.6 % of a value, and BF16 roundings of 2^-8: taken four times, each
    independent, an error of 6 % in the gradient and a cosine of 0.998."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    block = moe_step.ExpertBlock(256, 384, 4, 2, gen, quantized=False)
    x, res = moe_step.normal(gen, 512, 256, dtype=torch.bfloat16), moe_step.normal(gen, 512, 256, dtype=torch.bfloat16)
    mixed, h = block.forward(x, res)
    d = moe_step.normal(gen, 512, 256, sigma=1e-2, dtype=torch.bfloat16)
    dx = block.backward(d, torch.zeros_like(h))
    w = {n: v.clone().requires_grad_() for n, v in block.masters.items()}
    w["up"], w["down"] = (c.float().requires_grad_() for c in (block.up, block.down))
    hh = h.float().requires_grad_()
    y = hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + moe_step.EPS) * w["gamma"]
    ids, weights = block.saved[3], torch.softmax((y @ w["router"]).gather(1, block.saved[3]), 1)
    out = torch.zeros_like(hh)
    for e in range(4):
        part = torch.nn.functional.silu(y @ w["up"][e]) @ w["down"][e]
        out = out + part * (weights * (ids == e)).sum(1, keepdim=True)
    out.backward(d.float())
    cos = lambda a, b: float(torch.nn.functional.cosine_similarity(a.detach().flatten().float(), b.detach().flatten().float(), dim=0))  # noqa: E731
    assert cos(mixed, out) > 0.99
    for n in w:
        assert cos(block.grads[n], w[n].grad) > 0.99, n
    assert cos(dx, hh.grad) > 0.99


@pytest.mark.parametrize("quantized", [False, True])
def test_loss_falls(quantized):
    """Forty steps halve the distance to the teacher where the products are plain;
    quantized ones leave the error of their own rounding, and have to gain too."""
    losses = moe_step.train(tokens=512, hidden=256, inner=512, experts=4, k=2, steps=40, quantized=quantized)
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) < (0.9 if quantized else 0.7) * sum(losses[:5]), losses
