"""Limits of the row operators that no device is needed to show: what is
refused before any kernel's index could leave its range."""
import ctypes
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


@pytest.mark.parametrize("cols", [1 << 31, (1 << 32) + 32, 1 << 33])
def test_rows_of_the_experts_are_narrower_than_2_31(L, cols):
    """One row of so many columns is below 2^34 elements, and its elements are
    numbered in 32 bits."""
    p = fake()
    assert L.fq_moe_dispatch(p, fq.FQ_F8_NONE, None, 1, 1, cols, 1, p, p, p, None) == fq.FQ_ERR_SHAPE
    assert L.fq_moe_dispatch(p, fq.FQ_F8_MX, p, 1, 1, cols, 1, p, p, p, None) == fq.FQ_ERR_SHAPE
    assert L.fq_moe_combine(p, p, 1, 1, cols, 1, p, p, None) == fq.FQ_ERR_SHAPE
    assert L.fq_moe_combine_bwd(p, p, p, 1, 1, cols, 1, p, p, p, p, None) == fq.FQ_ERR_SHAPE
    assert "cols" in L.fq_last_error().decode()


@pytest.mark.parametrize("f8, tile", [(False, 4096), (True, 2048)])
def test_a_plan_has_fewer_tiles_than_its_grid_can_walk_over(L, f8, tile):
    """The kernel's walk adds the grid to a 32-bit tile number: the last number has
    to stay below 2^32 with that added, whatever the tensors' lengths."""
    each = (1 << 34) // tile                                     # tiles of the longest tensor

    def plan(tiles):
        lengths = [1 << 34] * (tiles // each) + ([tiles % each * tile] if tiles % each else [])
        array = (fq.FqAdamWTensor * len(lengths))()
        for t, n in zip(array, lengths):
            t.w, t.g, t.m, t.v, t.m_scale, t.v_scale, t.n = 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, n
        size = L.fq_adamw_plan_size(len(lengths))
        buf = (ctypes.c_uint8 * (size + 64))()
        at = ctypes.addressof(buf)
        return L.fq_adamw_plan(array, len(lengths), int(f8), at + -at % 64, size)

    assert plan((1 << 32) - 2) == fq.FQ_ERR_SHAPE
    assert "tiles" in L.fq_last_error().decode()
    assert plan((1 << 31) + 1) == fq.FQ_ERR_SHAPE
    assert plan(1 << 31) == fq.FQ_OK


def test_adamw_refuses_what_fp32_does_not_hold(L):
    """lr and eps are used in FP32: an lr or eps that is infinite there, or a positive
    eps that is 0 there, would make weights NaN that the formula leaves finite."""
    t = fq.FqAdamWTensor(w=0x1000, g=0x2000, m=0x3000, v=0x4000, n=0, lr_mult=1.0)

    def step(**fields):
        h = fq.FqAdamWHyper(**dict(dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1), **fields))
        return L.fq_adamw_step(ctypes.byref(h), ctypes.byref(t), 1, None)

    for bad in (dict(lr=1e39), dict(lr=-1e39), dict(eps=1e39), dict(eps=1e-60), dict(eps=2.0 ** -150)):
        assert step(**bad) == fq.FQ_ERR_DESC, bad
    for good in (dict(lr=3.4e38), dict(lr=-1.0), dict(eps=3.4e38), dict(eps=2.0 ** -149), dict(eps=0.0), dict(lr=1e-60)):
        assert step(**good) == fq.FQ_OK, good
