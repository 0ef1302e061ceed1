"""The norm of many rows just wider than a power of two, which take other lanes
than wide rows do: forward with five waves a row, backward with ten and with
more workgroups.  Against float64, with the error bounds of test_gpu_norm."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import step as oracle
from test_gpu_norm import EPS, U, bf, check_codes, f64, inputs
from test_gpu_norm_rows import check_backward, guarded

pytestmark = pytest.mark.gpu

# rows at the lengths where the launcher changes its mind, and widths on both
# sides of 2048, 2560, 4096 and 5120 and where a first chunk is shared
SHAPES = [(4110, 2041), (4099, 2047), (8200, 2047), (4098, 2049), (4081, 2056), (3641, 2305), (7300, 2305), (3277, 2560),
          (3276, 2560), (3290, 2553), (3290, 2554), (511, 2560), (512, 4089), (513, 4095), (513, 4096), (512, 4104),
          (511, 4104), (600, 5120), (600, 5113), (600, 5114), (3300, 5120)]


@pytest.mark.parametrize("rows, cols", SHAPES)
@pytest.mark.parametrize("stream", ["none", "bf16", "f32"])
def test_forward_of_many_rows(rows, cols, stream):
    x, res, gamma, h = inputs(rows, cols, stream, seed=cols, gamma_type=torch.bfloat16 if rows % 2 else torch.float32)
    y, around_y = guarded(rows, cols, torch.bfloat16)
    hg, around_h = guarded(rows, cols, torch.float32 if stream == "f32" else torch.bfloat16)
    rstd = torch.empty(rows, device=DEV)
    fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, h=None if res is None else hg, y=y, rstd=rstd)
    n, r = oracle.rmsnorm(h, f64(gamma), EPS)
    if res is not None:
        assert np.array_equal(f64(hg), h.astype(np.float64))
    assert np.all(np.abs(f64(rstd) - r) <= 64 * U * r)
    assert np.all(np.abs(f64(y) - n) <= (2.0 ** -8 + 64 * U) * np.abs(n))
    assert all((t == 7).all() for t in around_y + around_h)


@pytest.mark.parametrize("rows, cols", [(4090, 2080), (3277, 2560), (6600, 2560), (512, 4128), (513, 5120), (3300, 5088)])
@pytest.mark.parametrize("f8", [fq.FQ_F8_MX, fq.FQ_F8_ROW])
@pytest.mark.parametrize("stream", ["none", "bf16"])
def test_forward_of_many_rows_8bit(rows, cols, f8, stream):
    x, res, gamma, h = inputs(rows, cols, stream, seed=cols)
    n, _ = oracle.rmsnorm(h, f64(gamma), EPS)
    y, around = guarded(rows, cols, torch.bfloat16)
    _, codes, scales = fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, f8=f8, y=y)
    v = check_codes(n, codes, scales, f8, cols)
    half = 0.0 if f8 == fq.FQ_F8_MX else 2.0 ** -8 + U
    assert np.all(np.abs(f64(y) - v) <= half * np.abs(v))
    assert all((t == 7).all() for t in around)


@pytest.mark.parametrize("rows, cols", [(1, 4096 + 8), (5, 4095), (300, 5120), (300, 5119), (1024, 4095), (1500, 4500),
                                        (4098, 4095), (4100, 4104), (3280, 5120), (3290, 5113), (3300, 5114), (33000, 513),
                                        (8200, 2049), (4200, 4001), (16500, 1017), (640, 2880), (641, 2880), (640, 1000),
                                        (641, 1001), (640, 3001), (640, 6072), (640, 64), (641, 64), (639, 4104)])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_backward(rows, cols, stream):
    x, res, gamma, h = inputs(rows, cols, stream, seed=rows)
    wide = torch.float32 if stream == "f32" else torch.bfloat16
    hg = torch.tensor(h, device=DEV).to(wide)
    rstd = torch.tensor(oracle.rmsnorm(h, f64(gamma), EPS)[1], dtype=torch.float32, device=DEV)
    rng = np.random.default_rng(cols)
    dy = bf(rng.standard_normal((rows, cols)) * 1e-3).to(DEV)
    dres = bf(rng.standard_normal((rows, cols)) * 1e-3).to(DEV).to(wide)
    dh, around = guarded(rows, cols, wide)
    dx, around_x = guarded(rows, cols, torch.bfloat16)
    need = fq.lib().fq_rmsnorm_bwd_workspace_size(rows, cols)
    room = torch.full((need + 64,), 7, dtype=torch.uint8, device=DEV)
    _, dgamma = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, dres=dres, dh=dh, dx=dx, ws=room[:need])
    check_backward(dy, h, gamma, rstd, dres, dh, dgamma)
    assert torch.equal(dx, dh.to(torch.bfloat16))
    assert all((t == 7).all() for t in around + around_x) and (room[need:] == 7).all()
    alone, _ = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, dres=dres, need_dgamma=False)
    assert torch.equal(alone, dh)
