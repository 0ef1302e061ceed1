"""Refusals of the operators around the linears: every call fails validation
before it touches the device, with the documented status."""
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


def fake(addr=0x10000):
    return ctypes.c_void_p(addr)


ODD = fake(0x10008)
BIG = 1 << 31


def fwd(L, x=fake(), res=fake(), st=0, gamma=fake(), gt=1, eps=1e-5, rows=4, cols=64, f8=0, h=fake(), y=fake(),
        codes=None, scales=None, rstd=fake()):
    return L.fq_rmsnorm_fwd(x, res, st, gamma, gt, eps, rows, cols, f8, h, y, codes, scales, rstd, None)


def test_norm_forward(L):
    assert fwd(L, x=None) == fwd(L, gamma=None) == fwd(L, y=None) == fwd(L, h=None) == fq.FQ_ERR_NULL
    assert fwd(L, x=ODD) == fwd(L, res=ODD) == fwd(L, h=ODD) == fwd(L, y=ODD) == fq.FQ_ERR_ALIGN
    assert fwd(L, rstd=fake(0x10002)) == fq.FQ_ERR_ALIGN
    assert fwd(L, rows=0) == fwd(L, cols=0) == fwd(L, cols=32769) == fwd(L, rows=BIG) == fq.FQ_ERR_SHAPE
    assert fwd(L, rows=1 << 30, cols=32768) == fq.FQ_ERR_SHAPE
    assert fwd(L, st=2) == fwd(L, gt=-1) == fwd(L, f8=3) == fwd(L, eps=-1.0) == fq.FQ_ERR_DESC
    assert fwd(L, eps=float("nan")) == fq.FQ_ERR_DESC
    assert fwd(L, res=None) == fq.FQ_ERR_DESC                      # h without a residual
    assert fwd(L, codes=fake(), scales=fake()) == fq.FQ_ERR_DESC   # codes without f8
    assert fwd(L, f8=1, cols=48, codes=fake(), scales=fake()) == fq.FQ_ERR_SHAPE
    assert fwd(L, f8=1, y=None) == fq.FQ_ERR_NULL
    assert fwd(L, f8=2, codes=fake()) == fq.FQ_ERR_NULL            # codes without scales
    assert "scales" in L.fq_last_error().decode()


def bwd(L, dy=fake(), h=fake(), st=0, gamma=fake(), gt=1, rstd=fake(), dres=None, rows=4, cols=64, dh=fake(), dx=None,
        dgamma=fake(), ws=fake(), ws_bytes=1 << 30):
    return L.fq_rmsnorm_bwd(dy, h, st, gamma, gt, rstd, dres, rows, cols, dh, dx, dgamma, ws, ws_bytes, None)


def test_norm_backward(L):
    assert bwd(L, dy=None) == bwd(L, h=None) == bwd(L, rstd=None) == bwd(L, dh=None) == bwd(L, ws=None) == fq.FQ_ERR_NULL
    assert bwd(L, dres=ODD) == bwd(L, dx=ODD) == bwd(L, ws=ODD) == bwd(L, dgamma=fake(0x10001)) == fq.FQ_ERR_ALIGN
    need = L.fq_rmsnorm_bwd_workspace_size(4, 64)
    assert need >= 256 and bwd(L, ws_bytes=need - 1) == fq.FQ_ERR_WORKSPACE
    assert bwd(L, cols=40000) == bwd(L, rows=-1) == fq.FQ_ERR_SHAPE
    assert bwd(L, st=7) == fq.FQ_ERR_DESC
    assert L.fq_rmsnorm_bwd_workspace_size(0, 64) == 0


def sort(L, ids=fake(), T=10, k=2, E=4, align=1, rows=None, offsets=fake(), pos=fake(), src=fake(), ws=fake(), ws_bytes=1 << 30):
    rows = L.fq_moe_rows(T, k, E, align) if rows is None else rows
    return L.fq_moe_sort(ids, T, k, E, align, rows, offsets, pos, src, ws, ws_bytes, None)


def test_moe_sort(L):
    assert sort(L, ids=None) == sort(L, offsets=None) == sort(L, pos=None) == sort(L, src=None) == fq.FQ_ERR_NULL
    assert sort(L, pos=fake(0x10002)) == fq.FQ_ERR_ALIGN
    for bad in (dict(T=0), dict(k=0), dict(k=65), dict(E=0), dict(E=1025), dict(align=0), dict(align=1025),
                dict(T=1 << 30, k=2), dict(T=1 << 62, k=4)):
        assert sort(L, **bad) == fq.FQ_ERR_SHAPE, bad
    assert sort(L, rows=19) == sort(L, rows=BIG) == fq.FQ_ERR_SHAPE
    need = L.fq_moe_sort_workspace_size(10000, 4, 32)
    assert need > 0 and L.fq_moe_sort_workspace_size(10, 4, 32) == 0
    assert sort(L, T=10000, k=4, E=32, ws_bytes=need - 1) == fq.FQ_ERR_WORKSPACE
    assert sort(L, T=10000, k=4, E=32, ws=None) == fq.FQ_ERR_NULL


def test_moe_rows_is_what_the_segments_take_at_most(L):
    assert L.fq_moe_rows(10, 2, 4, 1) == 20
    assert L.fq_moe_rows(1, 1, 1024, 128) == 128
    assert L.fq_moe_rows(1, 4, 32, 128) == 512
    # 100 assignments over 3 experts: 34 + 33 + 33 in tiles of 16 is 48 * 3
    assert L.fq_moe_rows(100, 1, 3, 16) == 144
    with pytest.raises(fq.FqError):
        fq.moe_rows(10, 2, 4, 0)


def test_moe_rows_operators(L):
    def disp(x=fake(), f8=0, scales=None, T=4, k=2, cols=64, rows=8, pos=fake(), src=fake(), y=fake()):
        return L.fq_moe_dispatch(x, f8, scales, T, k, cols, rows, pos, src, y, None)

    def comb(y=fake(), w=None, T=4, k=2, cols=64, rows=8, pos=fake(), out=fake()):
        return L.fq_moe_combine(y, w, T, k, cols, rows, pos, out, None)

    def cbwd(dout=fake(), y=fake(), w=fake(), T=4, k=2, cols=64, rows=8, pos=fake(), src=fake(), dy=fake(), dw=fake()):
        return L.fq_moe_combine_bwd(dout, y, w, T, k, cols, rows, pos, src, dy, dw, None)

    for f in (disp, comb, cbwd):
        for bad in (dict(T=0), dict(k=65), dict(cols=12), dict(cols=0), dict(rows=0), dict(rows=BIG), dict(cols=1 << 34),
                    dict(T=1 << 29, cols=64)):
            assert f(**bad) == fq.FQ_ERR_SHAPE, (f, bad)
        assert f(y=None) == f(pos=None) == fq.FQ_ERR_NULL
        assert f(y=ODD) == f(pos=fake(0x10001)) == fq.FQ_ERR_ALIGN
    assert disp(f8=1) == disp(f8=2) == disp(src=None) == fq.FQ_ERR_NULL
    assert disp(f8=4) == disp(scales=fake()) == fq.FQ_ERR_DESC
    assert disp(f8=1, scales=fake(), cols=40) == fq.FQ_ERR_SHAPE
    assert cbwd(w=None) == cbwd(dw=None) == cbwd(src=None) == fq.FQ_ERR_NULL
    assert comb(w=fake(0x10002)) == fq.FQ_ERR_ALIGN


def test_adamw(L):
    def call(hyper=None, tensor=None, count=1, null=False):
        h = fq.FqAdamWHyper(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, state_type=0)
        t = fq.FqAdamWTensor(w=0x1000, g=0x2000, m=0x3000, v=0x4000, n=100, g_type=0, lr_mult=1.0)
        for k, v in (hyper or {}).items():
            setattr(h, k, v)
        for k, v in (tensor or {}).items():
            setattr(t, k, v)
        return L.fq_adamw_step(ctypes.byref(h), None if null else ctypes.byref(t), count, None)

    assert L.fq_adamw_step(None, None, 0, None) == fq.FQ_ERR_NULL
    assert call(null=True) == fq.FQ_ERR_NULL
    assert call(count=-1) == fq.FQ_ERR_SHAPE
    for bad in (dict(step=0), dict(step=1 << 32), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=float("inf")),
                dict(state_type=2), dict(reserved=1), dict(beta1=float("nan"))):
        assert call(hyper=bad) == fq.FQ_ERR_DESC, bad
    for name in ("w", "g", "m", "v"):
        assert call(tensor={name: 0}) == fq.FQ_ERR_NULL, name
        assert call(tensor={name: 0x1004}) == fq.FQ_ERR_ALIGN, name
    assert call(tensor=dict(w_bf16=0x1002)) == fq.FQ_ERR_ALIGN
    assert call(tensor=dict(n=-1)) == call(tensor=dict(n=(1 << 34) + 1)) == fq.FQ_ERR_SHAPE
    assert call(tensor=dict(g_type=2)) == call(tensor=dict(reserved=1)) == fq.FQ_ERR_DESC
    assert call(tensor=dict(weight_decay=float("nan"))) == fq.FQ_ERR_DESC
    assert call(hyper=dict(state_type=1)) == fq.FQ_ERR_NULL            # no scales
    assert call(hyper=dict(state_type=1), tensor=dict(m_scale=0x5000, v_scale=0x5002)) == fq.FQ_ERR_ALIGN
    assert call(hyper=dict(grad_scale=0x5001)) == fq.FQ_ERR_ALIGN
    # nothing to do: nothing is launched
    assert call(tensor=dict(n=0, w=0, g=0, m=0, v=0)) == fq.FQ_OK
    assert call(count=0, null=True) == fq.FQ_OK


def test_binding_refuses_host_and_mistyped_tensors(L):
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        fq.fq_rmsnorm_fwd(x, torch.ones(64), 1e-5)
    with pytest.raises(ValueError, match="bfloat16"):
        fq.fq_rmsnorm_fwd(x.float(), torch.ones(64), 1e-5, y=x)
    with pytest.raises(ValueError):
        fq.fq_rmsnorm_fwd(x, torch.ones(64), 1e-5, res=x.half())
    with pytest.raises(ValueError, match="int32"):
        fq.fq_moe_sort(torch.zeros((4, 2), dtype=torch.int64), 4)
    with pytest.raises(ValueError):
        fq.adamw_plan([fq.AdamWTensor(w=torch.zeros(4), g=torch.zeros(4), m=torch.zeros(4), v=torch.zeros(4))])
