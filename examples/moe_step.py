"""A quantization-aware training step of a mixture-of-experts block on one GPU.

    python3 examples/moe_step.py [--tokens T] [--hidden H] [--inner N] [--experts E] [--k K] [--steps S] [--bf16]

One step runs, as a training program would:
  * residual addition and norm of the tokens, with 8-bit rows for the experts
    and the values they stand for to the router (fq_rmsnorm_fwd);
  * tokens sorted by expert in segments that the quantized products take, and
    dispatched from their 8-bit rows (fq_moe_sort, fq_moe_dispatch);
  * every expert's two NVFP4 linears (fq_qlinear_fwd; with --bf16 plain products,
    to compare with), and the results back to the tokens with the router's
    weights (fq_moe_combine);
  * all of that backward (fq_moe_combine_bwd, fq_qlinear_bwd, fq_moe_combine as
    the dispatch's gradient, fq_rmsnorm_bwd);
  * AdamW over all parameters, the experts with 8-bit states, gradients clipped
    to a global norm on the device (fq_adamw_step).
The task is synthetic: a random teacher of the same shape, with plain products.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import fp4_block_quantization_fq_amd as fq  # noqa: E402

EPS = 1e-5
ALIGN = 128                       # rows of an expert's segment: what the backward products take


def normal(gen, *shape, sigma=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)


class ExpertBlock:
    """Parameters (FP32 masters with BF16 copies) and the buffers of a step."""

    def __init__(self, hidden, inner, experts, k, gen, quantized=True):
        self.quantized = quantized
        self.hidden, self.inner, self.experts, self.k = hidden, inner, experts, k
        self.masters = {"gamma": torch.ones(hidden, device="cuda"),
                        "router": normal(gen, hidden, experts, sigma=hidden ** -0.5),
                        "up": normal(gen, experts, hidden, inner, sigma=hidden ** -0.5),
                        "down": normal(gen, experts, inner, hidden, sigma=inner ** -0.5)}
        self.up, self.down = (self.masters[n].to(torch.bfloat16) for n in ("up", "down"))
        self.grads = {"gamma": torch.zeros(hidden, device="cuda"),
                      "router": torch.zeros(hidden, experts, device="cuda"),
                      "up": torch.zeros_like(self.up), "down": torch.zeros_like(self.down)}
        self.dx = fq.fq_desc_nvfp4()
        self.dw = fq.fq_desc_nvfp4(axis=fq.FQ_AXIS_COL)
        self.dg = fq.fq_desc_mxfp4(rounding=fq.FQ_ROUND_SR)
        flat = lambda n: (self.masters[n].view(-1), self.grads[n].view(-1))  # noqa: E731
        small, large = [], []
        for n in ("gamma", "router"):
            w, g = flat(n)
            small.append(fq.AdamWTensor(w=w, g=g, **fq.adamw_state(w.numel(), w.device)))
        for n, copy in (("up", self.up), ("down", self.down)):
            w, g = flat(n)
            large.append(fq.AdamWTensor(w=w, g=g, w_bf16=copy.view(-1), weight_decay=0.01,
                                        **fq.adamw_state(w.numel(), w.device, f8=True)))
        self.plans = fq.adamw_plan(small), fq.adamw_plan(large)
        self.step_number = 0

    def linear(self, x, w, y):
        if self.quantized:
            fq.fq_qlinear_fwd(self.dx, self.dw, x, w, y=y)
        else:
            torch.mm(x, w, out=y)

    def linear_bwd(self, x, w, dy, dx, dw, seed):
        if self.quantized:
            self.dg.seed = seed
            fq.fq_qlinear_bwd(self.dx, self.dw, self.dg, x, w, dy, dx=dx, dw=dw)
        else:
            torch.mm(dy, w.T, out=dx)
            torch.mm(x.T, dy, out=dw)

    def forward(self, x, res):
        h = torch.empty_like(res)
        y, rstd = torch.empty_like(x), torch.empty(x.shape[0], device=x.device)
        _, codes, scales = fq.fq_rmsnorm_fwd(x, self.masters["gamma"], EPS, res=res, h=h, f8=fq.FQ_F8_MX, y=y, rstd=rstd)
        logits = y.float() @ self.masters["router"]
        top, ids = logits.topk(self.k, dim=1)
        weights = torch.softmax(top, 1)
        q = fq.fq_moe_sort(ids.to(torch.int32), self.experts, ALIGN)
        rows = fq.fq_moe_dispatch(codes, q, f8=fq.FQ_F8_MX, scales=scales)
        offsets = q.offsets.tolist()              # the products' shapes are the host's
        pre = torch.empty((rows.shape[0], self.inner), dtype=torch.bfloat16, device=x.device)
        out = torch.empty_like(rows)
        act = torch.empty_like(pre)
        for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
            if a == b:
                continue
            self.linear(rows[a:b], self.up[e], pre[a:b])
            act[a:b] = torch.nn.functional.silu(pre[a:b].float())
            self.linear(act[a:b], self.down[e], out[a:b])
        mixed = fq.fq_moe_combine(out, q, weights)
        self.saved = (h, y, rstd, ids, weights, q, offsets, rows, pre, act, out)
        return mixed, h

    def backward(self, dmixed, dh):
        """Gradients of the parameters (into self.grads) and of x and res."""
        h, y, rstd, ids, weights, q, offsets, rows, pre, act, out = self.saved
        dout, dweights = fq.fq_moe_combine_bwd(dmixed, out, q, weights)
        drows = torch.zeros_like(rows)
        for g in ("up", "down"):
            self.grads[g].zero_()
        for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
            if a == b:
                continue
            seed = (self.step_number * self.experts + e) * 8
            dact = torch.empty_like(act[a:b])
            self.linear_bwd(act[a:b], self.down[e], dout[a:b], dact, self.grads["down"][e], seed)
            p = pre[a:b].float()
            s = torch.sigmoid(p)
            dpre = (dact.float() * (s * (1 + p * (1 - s)))).to(torch.bfloat16)
            self.linear_bwd(rows[a:b], self.up[e], dpre, drows[a:b], self.grads["up"][e], seed + 4)
        dtop = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
        dlogits = torch.zeros((y.shape[0], self.experts), device=y.device).scatter_(1, ids, dtop)
        torch.mm(y.float().T, dlogits, out=self.grads["router"])
        dy = fq.fq_moe_combine(drows, q).float() + dlogits @ self.masters["router"].T
        dx, _ = fq.fq_rmsnorm_bwd(dy.to(torch.bfloat16), h, self.masters["gamma"], rstd, dres=dh, dgamma=self.grads["gamma"])
        return dx

    def update(self, lr, clip=1.0):
        self.step_number += 1
        norm = torch.stack([g.float().norm() for g in self.grads.values()]).norm()
        scale = (clip / norm.clamp_min(clip)).reshape(1)
        for plan in self.plans:
            fq.fq_adamw_step(plan, lr=lr, step=self.step_number, beta2=0.95, grad_scale=scale, seed=self.step_number)


def train(tokens=1024, hidden=512, inner=1024, experts=8, k=2, steps=30, lr=2e-3, seed=0, quantized=True, say=None):
    """Losses of `steps` steps on a random teacher's outputs."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    teacher = ExpertBlock(hidden, inner, experts, k, gen, quantized=False)
    block = ExpertBlock(hidden, inner, experts, k, gen, quantized)
    # the student starts next to the teacher: the router finds the same experts
    for n in ("router", "up", "down"):
        block.masters[n].mul_(0.5).add_(teacher.masters[n], alpha=0.5)
    block.up.copy_(block.masters["up"])
    block.down.copy_(block.masters["down"])
    losses = []
    for step in range(steps):
        x = normal(gen, tokens, hidden, dtype=torch.bfloat16)
        res = normal(gen, tokens, hidden, dtype=torch.bfloat16)
        want, _ = teacher.forward(x, res)
        got, h = block.forward(x, res)
        diff = got.float() - want.float()
        loss = diff.square().mean()
        dmixed = (diff * (2.0 / diff.numel() * tokens)).to(torch.bfloat16)
        block.backward(dmixed, torch.zeros_like(h))
        block.update(lr)
        losses.append(loss)
        if say:
            say(f"step {step + 1}: loss {float(loss):.5f}")
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 2880), ("inner", 2880), ("experts", 32), ("k", 4), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--bf16", action="store_true")
    a = ap.parse_args()
    train(a.tokens, a.hidden, a.inner, a.experts, a.k, a.steps, quantized=not a.bf16, say=lambda s: print(s, flush=True))


if __name__ == "__main__":
    main()
