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
