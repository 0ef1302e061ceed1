"""AdamW in calls that stream (from 2^24 elements on), elements past 2^32, and
moments that are not finite.  FP32 states against the formula in float64 on the
device, with the error bounds of test_gpu_adamw; 8-bit states against the same
step in calls that do not stream, whose codes are checked one by one there."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
import oracle as philox
from gpu_util import DEV
from oracle import step as oracle
from test_gpu_adamw import HYPER, U, check_f8, copy_of, decoded, tensors

pytestmark = pytest.mark.gpu


def check_f32(before, after, scale=1.0, hyper=HYPER):
    """One tensor in float64 on the device."""
    b1, b2, step = hyper["beta1"], hyper["beta2"], hyper["step"]
    for t, got in zip(before, after):
        d = lambda v: v.double()  # noqa: E731
        lr, decay = hyper["lr"] * t.lr_mult, float(np.float32(t.weight_decay))
        g = d(t.g) * scale
        m, v = b1 * d(t.m) + (1 - b1) * g, b2 * d(t.v) + (1 - b2) * g * g
        root = v.sqrt() / (1 - b2 ** step) ** 0.5 + hyper["eps"]
        kept = d(t.w) * (1 - lr * decay)
        w = kept - lr / (1 - b1 ** step) * m / root
        size = d(t.m).abs() + g.abs()
        assert ((d(got.m) - m).abs() <= 4 * U * size + 1e-44).all()
        assert ((d(got.v) - v).abs() <= 6 * U * v + 1e-44).all()
        reach = lr / (1 - b1 ** step) * size / root
        assert ((d(got.w) - w).abs() <= 3 * U * d(t.w).abs() + 12 * U * ((w - kept).abs() + reach)).all()
        if t.w_bf16 is not None:
            assert torch.equal(got.w_bf16, got.w.to(torch.bfloat16))


def by_list(ts, f8, seed=0, scale=None):
    array = (fq.FqAdamWTensor * len(ts))()
    for s, t in zip(array, ts):
        s.n, s.lr_mult, s.weight_decay = t.w.numel(), t.lr_mult, t.weight_decay
        s.g_type = fq.FQ_TYPE_BF16 if t.g.dtype == torch.bfloat16 else fq.FQ_TYPE_F32
        for name in ("w", "w_bf16", "g", "m", "v", "m_scale", "v_scale"):
            v = getattr(t, name)
            setattr(s, name, None if v is None else v.data_ptr())
    h = fq.FqAdamWHyper(seed=seed, grad_scale=None if scale is None else scale.data_ptr(), state_type=int(f8), **HYPER)
    assert fq.lib().fq_adamw_step(ctypes.byref(h), array, len(ts), torch.cuda.current_stream().cuda_stream) == fq.FQ_OK


def equal(a, b, names=("w", "w_bf16", "m", "v", "m_scale", "v_scale")):
    for name in names:
        u, v = getattr(a, name), getattr(b, name)
        assert (u is None and v is None) or torch.equal(u, v), name


# streaming, just below it, and streaming only together; a tail in each
SIZES = [[(1 << 24) + 5], [(1 << 24) - 4099], [(1 << 23) + 1, (1 << 23) + 4094, 77]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("grads", ["bf16", "f32"])
def test_fp32_states(sizes, grads):
    before = tensors(sizes, grads, False, seed=2)
    plan, listed = ([copy_of(t) for t in before] for _ in range(2))
    scale = torch.tensor([0.5], device=DEV)
    fq.fq_adamw_step(fq.adamw_plan(plan), grad_scale=scale, **HYPER)
    check_f32(before, plan, scale=0.5)
    by_list(listed, False, scale=scale)
    for a, b in zip(plan, listed):
        equal(a, b)


@pytest.mark.parametrize("grads", ["bf16", "f32"])
def test_8bit_states(grads):
    """Two tensors stream together and not by themselves; an empty one keeps the
    second one's number."""
    before = tensors([(1 << 23) + 5, (1 << 23) + 4094], grads, True, seed=3)
    together, alone, listed = ([copy_of(t) for t in before] for _ in range(3))
    wide = [decoded(t) for t in before]
    fq.fq_adamw_step(fq.adamw_plan(together), seed=11, **HYPER)
    empty = tensors([0], grads, True)[0]
    for ts in ([alone[0]], [empty, alone[1]]):
        fq.fq_adamw_step(fq.adamw_plan(ts), seed=11, **HYPER)
    by_list(listed, True, seed=11)
    fq.fq_adamw_step(fq.adamw_plan(wide), **HYPER)
    for a, b, c, f in zip(together, alone, listed, wide):
        equal(a, b)
        equal(a, c)
        equal(a, f, ("w", "w_bf16"))


def test_8bit_codes_past_32_bit_offsets():
    """The last blocks of more than 2^32 elements, code by code."""
    n, tail = (1 << 32) + 131, 131
    w, g = torch.zeros(n, device=DEV), torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    t = fq.AdamWTensor(w=w, g=g, **fq.adamw_state(n, DEV, True))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    w[-tail:] = torch.randn(tail, generator=gen, device=DEV)
    g[-tail:] = torch.randn(tail, generator=gen, device=DEV).to(torch.bfloat16)
    wide = fq.AdamWTensor(w=w[-tail:].clone(), g=g[-tail:].clone(), **fq.adamw_state(tail, DEV))
    seed, hyper = 0x123456789AB, dict(HYPER, step=3)
    fq.fq_adamw_step(fq.adamw_plan([t]), seed=seed, **hyper)
    fq.fq_adamw_step(fq.adamw_plan([wide]), **hyper)
    assert torch.equal(w[-tail:], wide.w)
    words = np.concatenate([philox.philox4x32_10([c & 0xFFFFFFFF, c >> 32, 0, 3], [seed & 0xFFFFFFFF, seed >> 32])
                            for c in range((1 << 32) // 4, (n + 3) // 4)])[:tail].astype(np.int64)
    mc, ms = oracle.quantize_state(wide.m.cpu().numpy(), words & 0xFFFF, oracle.E4M3_MAX, oracle.E4M3, False)
    vc, vs = oracle.quantize_state(wide.v.cpu().numpy(), words >> 16, oracle.E5M2_MAX, oracle.E5M2, True)
    assert np.array_equal(t.m[-tail:].cpu().numpy(), mc) and np.array_equal(t.v[-tail:].cpu().numpy(), vc)
    assert np.array_equal(t.m_scale[-2:].cpu().numpy(), ms) and np.array_equal(t.v_scale[-2:].cpu().numpy(), vs)
    assert int(t.m[: 1 << 20].max()) == 0 and int(t.v[-tail - 200: -tail].max()) == 0


def test_8bit_moments_that_are_not_finite():
    """Codes and scales around infinities and NaN, one by one: the element itself,
    its neighbours under the same scale, whole blocks, a block's only finite one."""
    n = 128 * 6 + 3
    t = tensors([n], "f32", True, seed=5)[0]
    t.g[3], t.g[130], t.g[399] = float("inf"), float("nan"), -float("inf")
    t.g[401] = 1e25                               # finite, its square is not: v alone
    t.g[512:640] = float("nan")                   # a whole block
    t.g[640:767] = -float("inf")                  # all but one
    t.m[768] = 0x7F                               # a state that already was NaN
    t.v[769] = 0x7F
    wide = decoded(t)
    fq.fq_adamw_step(fq.adamw_plan([wide]), **HYPER)
    fq.fq_adamw_step(fq.adamw_plan([t]), seed=1, **HYPER)
    rm, rv = oracle.state_draws(n, 0, HYPER["step"], 1)
    with np.errstate(invalid="ignore"):
        mc, ms = oracle.quantize_state(wide.m.cpu().numpy(), rm, oracle.E4M3_MAX, oracle.E4M3, False)
        vc, vs = oracle.quantize_state(wide.v.cpu().numpy(), rv, oracle.E5M2_MAX, oracle.E5M2, True)
    m, v = wide.m.cpu(), wide.v.cpu()
    assert not torch.isfinite(m[[3, 130, 399, 768]]).any() and torch.isfinite(m[401]) and not torch.isfinite(v[[401, 769]]).any()
    assert np.array_equal(t.m_scale.cpu().numpy(), ms) and np.array_equal(t.v_scale.cpu().numpy(), vs)
    assert np.isfinite(ms).all() and np.isfinite(vs).all()
    got_m, got_v = t.m.cpu().numpy(), t.v.cpu().numpy()
    nan = np.isnan(m.numpy())                     # a NaN's sign is not defined
    assert np.array_equal(np.where(nan, got_m & 0x7F, got_m), np.where(nan, mc & 0x7F, mc))
    assert np.array_equal(got_v, vc)
    same = torch.isfinite(wide.w)
    assert torch.equal(t.w[same], wide.w[same]) and torch.equal(torch.isnan(t.w), torch.isnan(wide.w))
    assert torch.equal(torch.isfinite(t.w), same)


def test_a_short_weight_is_a_short_tensor():
    """The weight's length is the tensor's; what the other operands have beyond it
    stays as it was."""
    t = tensors([100], "bf16", False)[0]
    short = copy_of(t)
    short.w = t.w[:99].clone()
    fq.fq_adamw_step(fq.adamw_plan([short]), **HYPER)
    whole = copy_of(t)
    fq.fq_adamw_step(fq.adamw_plan([whole]), **HYPER)
    assert torch.equal(short.w, whole.w[:99]) and torch.equal(short.m[:99], whole.m[:99])
    for name in ("m", "v", "w_bf16"):
        assert torch.equal(getattr(short, name)[99:], getattr(t, name)[99:]), name
