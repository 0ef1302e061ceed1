"""The norm and its backward where a row's place matters: rows that start at any
element (widths that are no multiple of 8, each starting place, the widest),
walks of a group over several such rows, few rows against many, and more rows
than a grid takes.  Against float64, with the error bounds of test_gpu_norm."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import step as oracle
from test_gpu_norm import EPS, U, bf, f64, inputs

pytestmark = pytest.mark.gpu


def guarded(rows, cols, dtype):
    """A matrix inside a larger buffer of sevens, and the elements around it."""
    pad = 64
    buf = torch.full((rows * cols + 2 * pad,), 7.0, dtype=dtype, device=DEV)
    return buf[pad: pad + rows * cols].view(rows, cols), (buf[:pad], buf[pad + rows * cols:])


@pytest.mark.parametrize("cols", [1, 2, 3, 5, 9, 57, 58, 63, 65, 121, 122, 249, 250, 505, 506, 1017, 1018, 2041, 2042,
                                  4089, 4090, 4095, 8185, 8186, 16377, 16378, 32762, 32763, 32766, 32767])
@pytest.mark.parametrize("stream", ["none", "bf16", "f32"])
def test_any_width(cols, stream):
    rows = 19 if cols < 9000 else 9
    x, res, gamma, h = inputs(rows, cols, stream, seed=cols, gamma_type=torch.bfloat16 if cols % 2 else torch.float32)
    wide = torch.float32 if stream == "f32" else torch.bfloat16
    y, around_y = guarded(rows, cols, torch.bfloat16)
    hg, around_h = guarded(rows, cols, wide)
    rstd = torch.empty(rows, device=DEV)
    fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, h=None if res is None else hg, y=y, rstd=rstd)
    n, r = oracle.rmsnorm(h, f64(gamma), EPS)
    if res is None:
        hg = x
    assert np.array_equal(f64(hg), h.astype(np.float64))
    assert np.all(np.abs(f64(rstd) - r) <= 64 * U * r)
    assert np.all(np.abs(f64(y) - n) <= (2.0 ** -8 + 64 * U) * np.abs(n))
    assert all((t == 7).all() for t in around_y + around_h)
    rng = np.random.default_rng(cols)
    dy = bf(rng.standard_normal((rows, cols)) * 1e-3).to(DEV)
    dres = bf(rng.standard_normal((rows, cols)) * 1e-3).to(DEV).to(wide)
    dh, around = guarded(rows, cols, wide)
    dx, around_x = guarded(rows, cols, torch.bfloat16)
    _, dgamma = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, dres=dres, dh=dh, dx=dx)
    check_backward(dy, h, gamma, rstd, dres, dh, dgamma)
    assert torch.equal(dx, dh.to(torch.bfloat16))
    assert all((t == 7).all() for t in around + around_x)


def check_backward(dy, h, gamma, rstd, dres, dh, dgamma):
    rows = h.shape[0]
    r32 = f64(rstd)
    want, wg = oracle.rmsnorm_bwd(f64(dy), h, f64(gamma), r32, None if dres is None else f64(dres))
    xh, g = h * r32[:, None], f64(dy) * f64(gamma)
    size = r32[:, None] * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    fp32 = 80 * U * size + 2 * U * np.abs(want)
    half = U if dh.dtype == torch.float32 else 2.0 ** -8
    assert np.all(np.abs(f64(dh) - want) <= half * np.abs(want) + (1 + half) * fp32)
    assert np.all(np.abs(f64(dgamma) - wg) <= (rows + 8) * U * np.abs(f64(dy) * xh).sum(0) + 1e-30)


@pytest.mark.parametrize("rows, cols", [(40000, 53), (33000, 64), (9001, 123), (9000, 512), (4099, 1003), (1025, 2049),
                                        (1500, 2881), (2051, 4088), (530, 8189), (513, 16383), (300, 32767), (1024, 96),
                                        (1024, 4097), (1023, 2047), (700, 3001)])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_backward_over_many_rows(rows, cols, stream):
    x, res, gamma, h = inputs(rows, cols, stream, seed=rows)
    wide = torch.float32 if stream == "f32" else torch.bfloat16
    hg = torch.tensor(h, device=DEV).to(wide)
    rstd = torch.tensor(oracle.rmsnorm(h, f64(gamma), EPS)[1], dtype=torch.float32, device=DEV)
    rng = np.random.default_rng(cols)
    dy = bf(rng.standard_normal((rows, cols)) * 1e-3).to(DEV)
    dres = bf(rng.standard_normal((rows, cols)) * 1e-3).to(DEV).to(wide)
    dh, dgamma = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, dres=dres)
    check_backward(dy, h, gamma, rstd, dres, dh, dgamma)
    alone, _ = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, dres=dres, need_dgamma=False)
    assert torch.equal(alone, dh)


@pytest.mark.parametrize("rows, cols", [(64, 256), (64, 257), (3000, 64)])
def test_gradient_written_over_its_inputs(rows, cols):
    """dh over h, and over dy, gives what it gives elsewhere (the columns' sums
    need both inputs whole)."""
    x, res, gamma, h = inputs(rows, cols, "bf16", seed=1)
    hg = torch.tensor(h, device=DEV).to(torch.bfloat16)
    rstd = torch.tensor(oracle.rmsnorm(h, f64(gamma), EPS)[1], dtype=torch.float32, device=DEV)
    dy = bf(np.random.default_rng(3).standard_normal((rows, cols))).to(DEV)
    ws = fq.rmsnorm_bwd_workspace(rows, cols, DEV)
    want = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, ws=ws)
    for over in ("h", "dy"):
        h2, dy2 = hg.clone(), dy.clone()
        dh, dgamma = fq.fq_rmsnorm_bwd(dy2, h2, gamma, rstd, dh=h2 if over == "h" else dy2, ws=ws)
        assert torch.equal(dh, want[0])
        size = np.abs(f64(dy) * h * f64(rstd)[:, None]).sum(0)
        assert np.all(np.abs(f64(dgamma) - f64(want[1])) <= 2 * (rows + 8) * U * size)


def test_more_rows_than_a_grid_takes():
    rows, cols = (1 << 25) + (1 << 20) + 5, 8
    x = torch.randn((rows, cols), device=DEV).to(torch.bfloat16)
    gamma = torch.linspace(0.5, 2, cols, device=DEV)
    rstd = torch.empty(rows, device=DEV)
    _, y = fq.fq_rmsnorm_fwd(x, gamma, EPS, rstd=rstd)
    dh, dgamma = fq.fq_rmsnorm_bwd(y, x, gamma, rstd)
    some = torch.cat((torch.arange(40), torch.arange(rows // 2, rows // 2 + 40), torch.arange(rows - 40, rows))).to(DEV)
    n, r = oracle.rmsnorm(f64(x[some]), f64(gamma), EPS)
    assert np.all(np.abs(f64(y[some]) - n) <= (2.0 ** -8 + 64 * U) * np.abs(n))
    want, _ = oracle.rmsnorm_bwd(f64(y[some]), f64(x[some]), f64(gamma), f64(rstd[some]))
    g, xh = f64(y[some]) * f64(gamma), f64(x[some]) * f64(rstd[some])[:, None]
    size = f64(rstd[some])[:, None] * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    assert np.all(np.abs(f64(dh[some]) - want) <= 2.0 ** -8 * np.abs(want) + 82 * U * size)
    # sums of 33 M products of like sign: every column's at once, in float64
    total = torch.zeros(cols, dtype=torch.float64, device=DEV)
    for a in range(0, rows, 1 << 22):
        b = slice(a, a + (1 << 22))
        total += (y[b].double() * x[b].double() * rstd[b].double()[:, None]).sum(0)
    # each of 32768 walks adds 1056 products, then 65 and 576 sums are added
    assert np.all(np.abs(f64(dgamma) - f64(total)) <= 1800 * U * f64(total))
