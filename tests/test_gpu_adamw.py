"""AdamW over many tensors on the GPU.  FP32 states against float64: m and v
are three and four roundings of sums of like signs or of two terms, w six more
on the update.  8-bit states: the codes must be exactly those of the rounding
rule applied to the moments, which the FP32-state path computes from the same
decoded values."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import step as oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=1e-3, step=7, beta1=0.9, beta2=0.98, eps=1e-8)


def f64(t):
    return t.detach().cpu().double().numpy()


def tensors(sizes, grads, f8, seed=0, copies=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        w = torch.randn(n, generator=g, device=DEV) * 0.02
        grad = (torch.randn(n, generator=g, device=DEV) * 1e-2 * 3.0 ** torch.randn(n, generator=g, device=DEV))
        grad = grad if grads == "f32" or (grads == "mixed" and i % 2) else grad.to(torch.bfloat16)
        st = fq.adamw_state(n, DEV, f8)
        if f8:
            st["m"].random_(0, 256, generator=g)
            st["m"][(st["m"] & 0x7F) == 0x7F] = 0
            st["v"].random_(0, 0x7C, generator=g)
            st["m_scale"].uniform_(1e-6, 1e-4, generator=g)
            st["v_scale"].uniform_(1e-12, 1e-9, generator=g)
        else:
            st["m"] = torch.randn(n, generator=g, device=DEV) * 1e-3
            st["v"] = torch.rand(n, generator=g, device=DEV) * 1e-5
        out.append(fq.AdamWTensor(w=w, g=grad, w_bf16=torch.zeros(n, dtype=torch.bfloat16, device=DEV)
                                  if copies and i % 3 != 1 else None, weight_decay=0.1 * (i % 3),
                                  lr_mult=1.0 + 0.5 * (i % 2), **st))
    return out


def copy_of(t):
    new = {k: getattr(t, k) for k in t.__dataclass_fields__}
    return fq.AdamWTensor(**{k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in new.items()})


def check_f32(before, after, scale=1.0, hyper=HYPER):
    for t, got in zip(before, after):
        lr = hyper["lr"] * t.lr_mult
        w, m, v = oracle.adamw(f64(t.w), f64(t.g), f64(t.m), f64(t.v), lr=lr, step=hyper["step"], beta1=hyper["beta1"],
                               beta2=hyper["beta2"], eps=hyper["eps"], weight_decay=float(np.float32(t.weight_decay)), scale=scale)
        gs = np.abs(f64(t.g)) * abs(scale)
        assert np.all(np.abs(f64(got.m) - m) <= 4 * U * (np.abs(f64(t.m)) + gs) + 1e-44)
        assert np.all(np.abs(f64(got.v) - v) <= 6 * U * v + 1e-44)
        step = np.abs(w - f64(t.w) * (1 - lr * t.weight_decay))
        # m's error is relative to its terms, so the update's is too
        reach = lr / (1 - hyper["beta1"] ** hyper["step"]) * (np.abs(f64(t.m)) + gs) / (
            np.sqrt(v) / np.sqrt(1 - hyper["beta2"] ** hyper["step"]) + hyper["eps"])
        assert np.all(np.abs(f64(got.w) - w) <= 3 * U * np.abs(f64(t.w)) + 12 * U * (step + reach))
        if t.w_bf16 is not None:
            assert torch.equal(got.w_bf16, got.w.to(torch.bfloat16))


RAGGED = [1, 2, 7, 8, 9, 127, 128, 129, 255, 1000, 2047, 2048, 2049, 4096, 70001]


@pytest.mark.parametrize("grads", ["bf16", "f32", "mixed"])
def test_fp32_states(grads):
    before = tensors(RAGGED, grads, False)
    after = [copy_of(t) for t in before]
    fq.fq_adamw_step(fq.adamw_plan(after), **HYPER)
    check_f32(before, after)


@pytest.mark.parametrize("count", [1, 31, 32, 33, 64, 65, 300])
def test_many_tensors(count):
    """One, just under and over a launch's table, and many; empty ones among them."""
    sizes = [(i * 37) % 300 for i in range(count)]
    before = tensors(sizes, "mixed", False, seed=count)
    after = [copy_of(t) for t in before]
    fq.fq_adamw_step(fq.adamw_plan(after), **HYPER)
    check_f32([t for t in before if t.w.numel()], [t for t in after if t.w.numel()])


def test_no_tensors_and_only_empty_ones():
    fq.fq_adamw_step(fq.adamw_plan([]), **HYPER)
    fq.fq_adamw_step(fq.adamw_plan(tensors([0, 0], "bf16", False)), **HYPER)


def test_first_step_from_zero_state_and_gradient_scale():
    before = tensors([500], "f32", False)
    before[0].m.zero_()
    before[0].v.zero_()
    after = [copy_of(t) for t in before]
    hyper = dict(HYPER, step=1)
    fq.fq_adamw_step(fq.adamw_plan(after), grad_scale=torch.tensor([0.25], device=DEV), **hyper)
    check_f32(before, after, scale=0.25, hyper=hyper)


def decoded(t):
    """The same tensor with its moments in FP32."""
    n = t.w.numel()
    wide = lambda s: s.repeat_interleave(fq.STATE_BLOCK)[:n]  # noqa: E731
    m = t.m.view(torch.float8_e4m3fn).float() * wide(t.m_scale)
    v = t.v.view(torch.float8_e5m2).float() * wide(t.v_scale)
    c = copy_of(t)
    c.m, c.v, c.m_scale, c.v_scale = m, v, None, None
    return c


def check_f8(wide, after, seed, step, numbers=None):
    """`wide`: the FP32-state tensors after the step."""
    for i, (f, t) in enumerate(zip(wide, after)):
        n = t.w.numel()
        assert torch.equal(f.w, t.w)
        if t.w_bf16 is not None:
            assert torch.equal(f.w_bf16, t.w_bf16)
        rm, rv = oracle.state_draws(n, i if numbers is None else numbers[i], step, seed)
        mc, ms = oracle.quantize_state(f.m.cpu().numpy(), rm, oracle.E4M3_MAX, oracle.E4M3, False)
        vc, vs = oracle.quantize_state(f.v.cpu().numpy(), rv, oracle.E5M2_MAX, oracle.E5M2, True)
        assert np.array_equal(t.m_scale.cpu().numpy(), ms) and np.array_equal(t.v_scale.cpu().numpy(), vs)
        bad = np.flatnonzero(t.m.cpu().numpy() != mc)
        assert bad.size == 0, (i, n, bad[:5], t.m.cpu().numpy()[bad[:5]], mc[bad[:5]])
        bad = np.flatnonzero(t.v.cpu().numpy() != vc)
        assert bad.size == 0, (i, n, bad[:5], t.v.cpu().numpy()[bad[:5]], vc[bad[:5]])


@pytest.mark.parametrize("grads", ["bf16", "f32"])
def test_8bit_states(grads):
    after = tensors(RAGGED, grads, True)
    wide = [decoded(t) for t in after]
    seed = 0x1234567890ABCDEF
    fq.fq_adamw_step(fq.adamw_plan(wide), **HYPER)
    fq.fq_adamw_step(fq.adamw_plan(after), seed=seed, **HYPER)
    check_f8(wide, after, seed, HYPER["step"])


def test_8bit_states_number_of_the_tensor_counts_over_launches():
    sizes = [0 if i % 5 == 0 else 130 for i in range(80)]
    after = tensors(sizes, "bf16", True)
    wide = [decoded(t) for t in after]
    fq.fq_adamw_step(fq.adamw_plan(wide), **HYPER)
    fq.fq_adamw_step(fq.adamw_plan(after), seed=3, **HYPER)
    live = [i for i in range(80) if sizes[i]]
    check_f8([wide[i] for i in live], [after[i] for i in live], 3, HYPER["step"], numbers=live)


def test_8bit_zero_tiny_and_huge_blocks():
    """Zero state and gradient, values whose scale would be below the normal
    range, and values near the largest FP32."""
    n = 128 * 5
    t = fq.AdamWTensor(w=torch.ones(n, device=DEV), g=torch.zeros(n, device=DEV), **fq.adamw_state(n, DEV, True))
    t.g[128:256] = torch.linspace(-1e-19, 1e-19, 128, device=DEV)
    t.g[256:384] = 1e18
    t.g[384:512] = torch.logspace(-18, 0, 128, device=DEV)
    t.g[515] = 1e-4
    wide = decoded(t)
    hyper = dict(HYPER, step=1)
    fq.fq_adamw_step(fq.adamw_plan([wide]), **hyper)
    fq.fq_adamw_step(fq.adamw_plan([t]), seed=9, **hyper)
    check_f8([wide], [t], 9, 1)
    assert (t.m[:128] == 0).all() and (t.v[:128] == 0).all()
    assert ((wide.v > 0).cpu() == (t.v.cpu() > 0)).all()          # no positive v is lost


def test_8bit_not_finite_stays_with_its_element():
    n = 400
    t = tensors([n], "f32", True)[0]
    t.g[3], t.g[130], t.g[399] = float("inf"), float("nan"), -float("inf")
    wide = decoded(t)
    fq.fq_adamw_step(fq.adamw_plan([wide]), **HYPER)
    before = copy_of(t)
    fq.fq_adamw_step(fq.adamw_plan([t]), seed=1, **HYPER)
    bad = torch.zeros(n, dtype=torch.bool)
    bad[[3, 130, 399]] = True
    assert ((t.m.cpu() & 0x7F) == 0x7F)[bad].all() and (t.v.cpu() == 0x7F)[bad].all()
    assert not ((t.m.cpu() & 0x7F) == 0x7F)[~bad].any()
    assert torch.isfinite(t.w.cpu()[~bad]).all() and torch.isfinite(t.m_scale).all()
    assert before.m_scale.shape == t.m_scale.shape


def test_8bit_training_follows_fp32():
    """A least-squares problem: after 200 steps both reach a small loss, the
    8-bit run within a factor of 3 of the FP32 one."""
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    a = torch.randn((256, 64), generator=g, device=DEV)
    target = torch.randn((64, 40), generator=g, device=DEV)
    loss = {}
    for f8 in (False, True):
        w, grad = torch.zeros(64 * 40, device=DEV), torch.zeros(64 * 40, device=DEV)
        plan = fq.adamw_plan([fq.AdamWTensor(w=w, g=grad, **fq.adamw_state(w.numel(), DEV, f8))])
        for step in range(1, 201):
            e = a @ (w.view(64, 40) - target)
            grad.copy_((a.T @ e).reshape(-1) / 256)
            fq.fq_adamw_step(plan, lr=0.05, step=step, seed=5)
        loss[f8] = float((a @ (w.view(64, 40) - target)).square().mean())
    assert loss[False] < 0.05 and loss[True] < 3 * loss[False] + 0.02, loss


def test_another_stream_and_graph():
    before = tensors([5000, 77], "bf16", True)
    want = [copy_of(t) for t in before]
    fq.fq_adamw_step(fq.adamw_plan(want), seed=2, **HYPER)
    fq.fq_adamw_step(fq.adamw_plan(want), seed=2, **HYPER)
    got = [copy_of(t) for t in before]
    plan = fq.adamw_plan(got)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fq.fq_adamw_step(plan, seed=2, stream=side, **HYPER)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        fq.fq_adamw_step(plan, seed=2, **HYPER)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.w, b.w) and torch.equal(a.m, b.m) and torch.equal(a.v, b.v)
        assert torch.equal(a.m_scale, b.m_scale)


def test_beyond_32_bit_offsets():
    n = (1 << 32) + 131
    w = torch.zeros(n, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g[-5:], w[-5:] = 0.5, 1.0
    t = fq.AdamWTensor(w=w, g=g, **fq.adamw_state(n, DEV, True))
    fq.fq_adamw_step(fq.adamw_plan([t]), lr=0.1, step=1, seed=4)
    assert torch.allclose(w[-5:], torch.full((5,), 0.9, device=DEV), atol=1e-6)
    assert float(w[:1000].abs().max()) == 0 and float(w[-6]) == 0
    assert (t.v[-5:] > 0).all() and int(t.v[-6]) == 0
    m = t.m[-5:].view(torch.float8_e4m3fn).float() * t.m_scale[-1]
    assert torch.allclose(m, torch.full((5,), 0.05, device=DEV), rtol=1e-6)
