"""AdamW plans without a device: what they refuse, and that an empty one is a
step that launches nothing."""
import ctypes
import os

import pytest
import torch

import fp4_block_quantization_fq_amd as fq


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fq.LIB_PATH):
        pytest.skip("libfq.so not built")
    return fq.lib()


def make(L, n=100, state_type=0, count=1, nbytes=None, null=False, **fields):
    t = fq.FqAdamWTensor(w=0x1000, g=0x2000, m=0x3000, v=0x4000, n=n, g_type=0, lr_mult=1.0)
    for k, v in fields.items():
        setattr(t, k, v)
    buf = torch.empty(4096, dtype=torch.uint8)
    nbytes = L.fq_adamw_plan_size(count) if nbytes is None else nbytes
    return L.fq_adamw_plan(ctypes.byref(t), count, state_type, None if null else buf.data_ptr(), nbytes), buf


def hyper(**fields):
    h = fq.FqAdamWHyper(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, state_type=0)
    for k, v in fields.items():
        setattr(h, k, v)
    return ctypes.byref(h)


def test_plan_size(L):
    assert L.fq_adamw_plan_size(-1) == 0 and L.fq_adamw_plan_size(1 << 31) == 0
    assert 0 < L.fq_adamw_plan_size(0) < L.fq_adamw_plan_size(1) < L.fq_adamw_plan_size(200)


def test_plan_refusals(L):
    assert make(L)[0] == fq.FQ_OK
    assert make(L, null=True)[0] == fq.FQ_ERR_NULL
    assert make(L, nbytes=L.fq_adamw_plan_size(1) - 1)[0] == fq.FQ_ERR_WORKSPACE
    assert make(L, state_type=2)[0] == fq.FQ_ERR_DESC
    assert make(L, w=0)[0] == fq.FQ_ERR_NULL and make(L, m=0x3004)[0] == fq.FQ_ERR_ALIGN
    assert make(L, state_type=1)[0] == fq.FQ_ERR_NULL              # no scales
    assert make(L, n=-1)[0] == fq.FQ_ERR_SHAPE
    assert make(L, weight_decay=float("inf"))[0] == fq.FQ_ERR_DESC


def test_step_refusals(L):
    ok, plan = make(L)
    step = lambda h=hyper(), p=plan.data_ptr(), d=None: L.fq_adamw_step_plan(h, p, d, None)  # noqa: E731
    assert ok == fq.FQ_OK
    assert step() == fq.FQ_ERR_NULL                                # no copy on the device
    assert step(d=0x1008) == fq.FQ_ERR_ALIGN
    assert step(p=None) == fq.FQ_ERR_NULL
    assert step(h=None) == fq.FQ_ERR_NULL
    assert step(h=hyper(step=0), d=0x1000) == fq.FQ_ERR_DESC
    assert step(h=hyper(state_type=1), d=0x1000) == fq.FQ_ERR_DESC         # another plan's states
    assert step(p=torch.zeros(4096, dtype=torch.uint8).data_ptr(), d=0x1000) == fq.FQ_ERR_DESC
    empty = make(L, n=0, w=0)[1]
    assert step(p=empty.data_ptr()) == fq.FQ_OK


def test_binding_refuses_what_is_no_tensor(L):
    with pytest.raises(TypeError):
        fq._binding().rmsnorm_fwd(1, 2, 3)
    with pytest.raises(TypeError):
        fq.fq_rmsnorm_fwd([[1.0]], torch.ones(1), 1e-5, y=1)
    with pytest.raises(ValueError, match="matrix"):
        fq.fq_moe_dispatch(torch.ones(4), fq.MoeSorted(None, torch.zeros((4, 1), dtype=torch.int32),
                                                       torch.zeros(4, dtype=torch.int32)), y=torch.ones(4))
    with pytest.raises(ValueError):
        fq.fq_rmsnorm_fwd(torch.ones((2, 8)).to_sparse(), torch.ones(8), 1e-5, y=torch.ones((2, 8)))
