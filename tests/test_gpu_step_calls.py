"""Calls of the row operators: what the binding refuses beside what the library
does, calls on a stream of their own that allocate for themselves, and the two
ways to an AdamW step."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from test_gpu_adamw import HYPER, copy_of, decoded, tensors

pytestmark = pytest.mark.gpu


def bf(*shape):
    return torch.ones(shape, dtype=torch.bfloat16, device=DEV)


def test_norm_refusals():
    x, gamma = bf(4, 64), torch.ones(64, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        fq.fq_rmsnorm_fwd(bf(4, 128)[:, ::2], gamma, 1e-5, y=x)
    with pytest.raises(ValueError, match="GPU"):
        fq.fq_rmsnorm_fwd(x, gamma.cpu(), 1e-5)
    with pytest.raises(ValueError, match="64 are needed"):
        fq.fq_rmsnorm_fwd(x, gamma[:63].contiguous(), 1e-5)
    with pytest.raises(ValueError, match="256 are needed"):
        fq.fq_rmsnorm_fwd(x, gamma, 1e-5, y=bf(3, 64))
    with pytest.raises(ValueError, match="float32"):
        fq.fq_rmsnorm_fwd(x, gamma, 1e-5, rstd=bf(4))
    with pytest.raises(ValueError, match="matrix"):
        fq.fq_rmsnorm_fwd(bf(64), gamma, 1e-5)
    with pytest.raises(TypeError):
        fq.fq_rmsnorm_fwd(x, [1.0] * 64, 1e-5)
    with pytest.raises(ValueError, match="1-byte|1"):
        fq.fq_rmsnorm_fwd(x, gamma, 1e-5, f8=fq.FQ_F8_MX, codes=torch.empty((4, 64), device=DEV))
    with pytest.raises(fq.FqError) as e:
        fq.fq_rmsnorm_fwd(bf(4, 48), torch.ones(48, device=DEV), 1e-5, f8=fq.FQ_F8_MX)
    assert e.value.status == fq.FQ_ERR_SHAPE
    with pytest.raises(fq.FqError) as e:
        fq.fq_rmsnorm_fwd(x.view(-1)[1:129].view(2, 64), gamma, 1e-5)
    assert e.value.status == fq.FQ_ERR_ALIGN
    rstd = torch.ones(4, device=DEV)
    with pytest.raises(ValueError, match="bfloat16"):
        fq.fq_rmsnorm_bwd(x, x, gamma, rstd, dres=torch.ones((4, 64), device=DEV))
    with pytest.raises(fq.FqError) as e:
        fq.fq_rmsnorm_bwd(x, x, gamma, rstd, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == fq.FQ_ERR_WORKSPACE


def test_moe_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    q = fq.fq_moe_sort(ids, 4)
    x, w = bf(4, 64), torch.ones((4, 2), device=DEV)
    with pytest.raises(ValueError, match="4 tokens were sorted"):
        fq.fq_moe_dispatch(bf(5, 64), q)
    with pytest.raises(ValueError, match="512 are needed"):
        fq.fq_moe_dispatch(x, q, y=bf(7, 64))
    with pytest.raises(ValueError, match="8 are needed"):
        fq.fq_moe_combine(bf(8, 64), q, w[:3].contiguous())
    with pytest.raises(ValueError, match="512 are needed"):
        fq.fq_moe_combine(bf(7, 64), q, w)
    with pytest.raises(fq.FqError) as e:
        fq.fq_moe_combine(bf(8, 60), q, w)
    assert e.value.status == fq.FQ_ERR_SHAPE
    with pytest.raises(ValueError, match="int32"):
        fq.fq_moe_combine(bf(8, 64), fq.MoeSorted(q.offsets, q.pos.long(), q.src), w)
    with pytest.raises(ValueError, match="5 are needed"):
        fq.fq_moe_sort(ids, 4, out=fq.MoeSorted(q.offsets[:4].contiguous(), q.pos, q.src))
    with pytest.raises(fq.FqError) as e:
        fq.fq_moe_sort(ids, 4, out=fq.MoeSorted(q.offsets, q.pos, q.src[:7].contiguous()))
    assert e.value.status == fq.FQ_ERR_SHAPE
    with pytest.raises(ValueError, match="512 are needed"):
        fq.fq_moe_combine_bwd(x, bf(8, 64), q, w, dy=bf(4, 64))


def test_adamw_refusals():
    t = tensors([100], "bf16", False)[0]
    plan = fq.adamw_plan([t])
    with pytest.raises(fq.FqError) as e:
        fq.fq_adamw_step(plan, lr=1e-3, step=0)
    assert e.value.status == fq.FQ_ERR_DESC
    with pytest.raises(ValueError, match="float32"):
        fq.fq_adamw_step(plan, lr=1e-3, step=1, grad_scale=bf(1))
    for name in ("w", "g", "m", "v", "w_bf16"):
        short = copy_of(t)
        setattr(short, name, getattr(t, name)[:99].contiguous())
        if name != "w":
            with pytest.raises(ValueError, match=name):
                fq.adamw_plan([short])


def test_list_and_plan_give_the_same_bits():
    sizes = [(i * 977) % 5000 for i in range(70)] + [0, 4096, 8191, 2048]
    for f8 in (False, True):
        a = tensors(sizes, "mixed", f8, seed=4)
        b = [copy_of(t) for t in a]
        scale = torch.tensor([0.5], device=DEV)
        fq.fq_adamw_step(fq.adamw_plan(a), grad_scale=scale, seed=77, **HYPER)
        array = (fq.FqAdamWTensor * len(b))()
        for s, t in zip(array, b):
            s.n, s.lr_mult, s.weight_decay = t.w.numel(), t.lr_mult, t.weight_decay
            s.g_type = fq.FQ_TYPE_BF16 if t.g.dtype == torch.bfloat16 else fq.FQ_TYPE_F32
            for name in ("w", "w_bf16", "g", "m", "v", "m_scale", "v_scale"):
                v = getattr(t, name)
                setattr(s, name, None if v is None else v.data_ptr())
        h = fq.FqAdamWHyper(seed=77, grad_scale=scale.data_ptr(), state_type=int(f8), **HYPER)
        st = fq.lib().fq_adamw_step(ctypes.byref(h), array, len(b), torch.cuda.current_stream().cuda_stream)
        assert st == fq.FQ_OK
        for s, t in zip(a, b):
            for name in ("w", "w_bf16", "m", "v", "m_scale", "v_scale"):
                u, v = getattr(s, name), getattr(t, name)
                assert (u is None and v is None) or torch.equal(u, v), name


def test_states_of_any_size_of_gradient():
    """Gradients from 1e-25 to 1e17, whose squares leave FP32's normal range and
    the range of the fast root: each against float64."""
    from oracle import step as oracle
    g = torch.logspace(-25, 17, 4001, device=DEV) * torch.where(torch.arange(4001, device=DEV) % 2 == 0, 1.0, -1.0)
    for eps in (1e-8, 1e-30):
        t = fq.AdamWTensor(w=torch.zeros(4001, device=DEV), g=g, **fq.adamw_state(4001, DEV))
        fq.fq_adamw_step(fq.adamw_plan([t]), lr=1.0, step=1, beta1=0.5, beta2=0.5, eps=eps)
        m, v = t.m.cpu().double().numpy(), t.v.cpu().double().numpy()
        want = -2 * m / (np.sqrt(v) * np.sqrt(2) + float(np.float32(eps)))
        # from the stored m and v: root and reciprocal within 2^-23 each, five roundings
        u = 2.0 ** -24
        assert np.all(np.abs(t.w.cpu().double().numpy() - want) <= 10 * u * np.abs(want) + 1e-44)
        wm = 0.5 * g.cpu().double().numpy()
        assert np.all(np.abs(m - wm) <= 2 * u * np.abs(wm) + 2e-45)
        wv = 0.5 * g.cpu().double().numpy() ** 2
        assert np.all(np.abs(v - wv) <= 4 * u * wv + 3e-45)


def test_calls_that_allocate_on_a_stream_of_their_own():
    """Outputs and workspaces made by a call on another stream stay whole while
    the current stream allocates and writes."""
    side = torch.cuda.Stream()
    x, gamma = torch.randn((4096, 2880), device=DEV).to(torch.bfloat16), torch.ones(2880, device=DEV)
    ids = torch.randint(0, 32, (4096, 4), dtype=torch.int32, device=DEV)
    rstd = torch.empty(4096, device=DEV)

    def work(stream):
        _, y = fq.fq_rmsnorm_fwd(x, gamma, 1e-5, rstd=rstd, stream=stream)
        dh, dgamma = fq.fq_rmsnorm_bwd(y, x, gamma, rstd, stream=stream)
        q = fq.fq_moe_sort(ids, 32, 64, stream=stream)
        r = fq.fq_moe_dispatch(y, q, stream=stream)
        return y, dh, dgamma, q.offsets, q.pos, q.src, r, fq.fq_moe_combine(r, q, stream=stream)

    want = [t.clone() for t in work(None)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got.append(work(side))
        for n in (2880, 64 << 10, 4096 * 2880 * 2):
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xAB)
    side.synchronize()
    torch.cuda.synchronize()
    for ts in got:
        assert all(torch.equal(a, b) for a, b in zip(ts, want))
