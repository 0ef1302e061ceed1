"""Refusals of the feed-forward products and of the 8-bit rows: every call fails
validation before it touches the device, with the documented status."""
import ctypes
import math
import os

import pytest

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


def linear(L, x=fake(), w=fake(), bias=fake(), bt=1, res=fake(), rows=4, k=64, n=64, experts=0, offsets=None, act=0, pre=None, pf8=0,
           ps=None, y=fake(), yt=0, ws=fake(), wb=1 << 40):
    return L.fq_linear_fwd(x, w, bias, bt, res, rows, k, n, experts, offsets, act, pre, pf8, ps, y, yt, ws, wb, None)


def glu(L, gate=fq.FqGate(fq.FQ_ACT_SILU, 1.0, math.inf, 0.0), x=fake(), w=fake(), bias=fake(), bt=1, rows=4, k=64, n=64, experts=0,
        offsets=None, pre=None, pf8=0, ps=None, y=fake(), ws=fake(), wb=1 << 40):
    return L.fq_glu_fwd(gate, x, w, bias, bt, rows, k, n, experts, offsets, pre, pf8, ps, y, ws, wb, None)


def linear_bwd(L, dy=fake(), x=fake(), xf8=0, xs=None, w=fake(), pre=fake(), pf8=0, ps=None, rows=4, k=64, n=64, experts=0, offsets=None,
               act=2, dx=fake(), dw=fake(), dwt=0, db=fake(), ws=fake(), wb=1 << 40):
    return L.fq_linear_bwd(dy, x, xf8, xs, w, pre, pf8, ps, rows, k, n, experts, offsets, act, dx, dw, dwt, db, ws, wb, None)


def glu_bwd(L, gate=fq.FqGate(fq.FQ_ACT_SILU, 1.0, math.inf, 0.0), dy=fake(), x=fake(), xf8=0, xs=None, w=fake(), pre=fake(), pf8=0,
            ps=None, rows=4, k=64, n=64, experts=0, offsets=None, dx=fake(), dw=fake(), dwt=0, db=fake(), h=fake(), ws=fake(), wb=1 << 40):
    return L.fq_glu_bwd(gate, dy, x, xf8, xs, w, pre, pf8, ps, rows, k, n, experts, offsets, dx, dw, dwt, db, h, ws, wb, None)


@pytest.mark.parametrize("call", [linear, glu, linear_bwd, glu_bwd])
def test_shapes(L, call):
    for bad in (dict(rows=0), dict(rows=-1), dict(rows=BIG), dict(rows=(1 << 30) + 1, k=8, n=8), dict(k=0), dict(k=4), dict(k=60), dict(n=0), dict(n=12), dict(k=-64),
                dict(k=(1 << 20) + 8), dict(n=(1 << 20) + 8), dict(rows=1 << 30, k=64), dict(rows=1 << 30, n=64),
                dict(k=1 << 20, n=1 << 20), dict(experts=1025, offsets=fake()), dict(experts=-1, offsets=fake()),
                dict(experts=1024, offsets=fake(), k=1 << 16, n=1 << 16), dict(rows=BIG - 1, k=1 << 20)):
        assert call(L, **bad) == fq.FQ_ERR_SHAPE, bad
    assert call(L, experts=3) == call(L, offsets=fake()) == fq.FQ_ERR_NULL
    assert call(L, experts=3, offsets=fake(0x10002)) == fq.FQ_ERR_ALIGN


@pytest.mark.parametrize("call", [linear, glu])
def test_forward(L, call):
    assert call(L, x=None) == call(L, w=None) == call(L, y=None) == fq.FQ_ERR_NULL
    assert call(L, x=ODD) == call(L, w=ODD) == call(L, bias=ODD) == call(L, y=ODD) == call(L, pre=ODD) == fq.FQ_ERR_ALIGN
    assert call(L, bt=2) == call(L, pre=fake(), pf8=2) == call(L, pre=fake(), pf8=3) == fq.FQ_ERR_DESC
    assert call(L, pre=fake(), pf8=1) == fq.FQ_ERR_NULL                     # codes without scales
    assert call(L, pre=fake(), ps=fake()) == call(L, ps=fake()) == fq.FQ_ERR_DESC
    assert call(L, pre=fake(), pf8=1, ps=fake(), n=40) == fq.FQ_ERR_SHAPE
    assert call(L, pre=fake(), pf8=1, ps=ODD) == fq.FQ_ERR_ALIGN


def test_linear(L):
    assert linear(L, act=-1) == linear(L, act=4) == linear(L, yt=2) == fq.FQ_ERR_DESC
    assert linear(L, res=ODD) == fq.FQ_ERR_ALIGN


@pytest.mark.parametrize("call", [glu, glu_bwd])
def test_gate(L, call):
    assert call(L, gate=None) == fq.FQ_ERR_NULL
    for bad in ((5, 1, 1, 0), (-1, 1, 1, 0), (2, math.inf, 1, 0), (2, math.nan, 1, 0), (3, 1.5, 1, 0), (0, 2.0, 1, 0), (2, 1, 0, 0),
                (2, 1, -1, 0), (2, 1, math.nan, 0), (2, 1, 1, math.inf), (2, 1, 1, math.nan)):
        assert call(L, gate=fq.FqGate(*bad)) == fq.FQ_ERR_DESC, bad


@pytest.mark.parametrize("call", [linear_bwd, glu_bwd])
def test_backward(L, call):
    assert call(L, dy=None) == call(L, x=None) == call(L, w=None) == call(L, pre=None) == call(L, ws=None) == fq.FQ_ERR_NULL
    assert call(L, dx=None, dw=None, db=None, **(dict(h=None) if call is glu_bwd else {})) == fq.FQ_ERR_NULL
    for name in ("dy", "x", "w", "pre", "dx", "dw", "db", "ws"):
        assert call(L, **{name: ODD}) == fq.FQ_ERR_ALIGN, name
    assert call(L, dwt=2) == call(L, xf8=3) == call(L, pf8=2) == call(L, xs=fake()) == call(L, ps=fake()) == fq.FQ_ERR_DESC
    assert call(L, xf8=1) == call(L, xf8=2) == call(L, pf8=1) == fq.FQ_ERR_NULL
    assert call(L, xf8=1, xs=fake(), k=72) == call(L, pf8=1, ps=fake(), n=72) == fq.FQ_ERR_SHAPE
    size = L.fq_linear_bwd_workspace_size if call is linear_bwd else L.fq_glu_bwd_workspace_size
    for f8, more in ((0, {}), (1, dict(xf8=1, xs=fake()))):
        need = size(4, 64, 64, 0, f8)
        assert need > 0 and call(L, wb=need - 1, **more) == fq.FQ_ERR_WORKSPACE
    assert size(4, 64, 64, 0, 1) > size(4, 64, 64, 0, 0)
    assert size(0, 64, 64, 0, 0) == size(4, 60, 64, 0, 0) == size(4, 64, 64, 0, 7) == size(4, 64, 64, -1, 0) == 0


def test_forward_workspaces(L):
    for size in (L.fq_linear_fwd_workspace_size, L.fq_glu_fwd_workspace_size):
        assert size(0, 64, 64, 0) == size(4, 60, 64, 0) == size(4, 64, 64, 1025) == 0
        # none of them overflows or grows beyond a few times its operands
        for rows, k, n, e in ((1, 8, 8, 0), (1, 1 << 20, 8, 0), (1 << 24, 64, 64, 1024), (4096, 4096, 4096, 0)):
            assert 0 <= size(rows, k, n, e) <= 4 * (64 << 20) + 64 * rows * n


def test_f8(L):
    def enc(x=fake(), f8=1, rows=4, cols=64, codes=fake(), scales=fake()):
        return L.fq_f8_encode(x, f8, rows, cols, codes, scales, None)

    def dec(codes=fake(), scales=fake(), f8=1, rows=4, cols=64, y=fake()):
        return L.fq_f8_decode(codes, scales, f8, rows, cols, y, None)

    for call, third in ((enc, "x"), (dec, "y")):
        for name in ("codes", "scales", third):
            assert call(**{name: None}) == fq.FQ_ERR_NULL
            assert call(**{name: ODD}) == fq.FQ_ERR_ALIGN
        assert call(f8=0) == call(f8=3) == fq.FQ_ERR_DESC
        for bad in (dict(rows=0), dict(cols=0), dict(cols=48), dict(rows=BIG), dict(cols=BIG), dict(rows=1 << 30, cols=64)):
            assert call(**bad) == fq.FQ_ERR_SHAPE, bad
    assert enc(f8=2, cols=32800) == fq.FQ_ERR_SHAPE
