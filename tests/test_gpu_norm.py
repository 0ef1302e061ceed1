"""Residual addition + root-mean-square norm and its backward on the GPU
against float64.

Error bounds, u = 2^-24 (half a step of FP32, relative): the sum of squares of
a row is at most 32 additions in a lane and 22 across lanes and waves, its root
halves that, and six further operations lead to n, so n is within 64 u of the
formula; a BF16 output adds half a step, 2^-8 of the value; an E4M3 one 2^-4 of
it or half the smallest step, 2^-10 of the scale."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import step as oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
WIDTHS = [1, 7, 8, 31, 96, 512, 513, 1000, 1032, 2048, 2880, 2881, 4096, 4100, 8192, 8200, 16384,
          16416, 32761, 32768]


def bf(a):
    return torch.tensor(np.asarray(a, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def inputs(rows, cols, stream, seed=0, gamma_type=torch.float32):
    rng = np.random.default_rng(seed)
    x = bf(rng.standard_normal((rows, cols)))
    res = None
    if stream != "none":
        r = rng.standard_normal((rows, cols)) * 2
        r[:, rng.integers(0, cols, 2)] *= 50
        res = bf(r) if stream == "bf16" else torch.tensor(r, dtype=torch.float32)
    gamma = torch.tensor(1 + 0.2 * rng.standard_normal(cols), dtype=torch.float32).to(gamma_type)
    h = f64(x).astype(np.float32) if res is None else oracle.residual(f64(x), f64(res), stream == "bf16")
    return x.to(DEV), None if res is None else res.to(DEV), gamma.to(DEV), h


def check_codes(n, codes, scales, f8, cols):
    """Codes and scales of 8-bit rows against the float64 values n; returns the
    values they stand for."""
    rows = n.shape[0]
    codes = codes.cpu().numpy()
    width = 32 if f8 == fq.FQ_F8_MX else cols
    amax = np.abs(n).reshape(rows, -1, width).max(2)
    if f8 == fq.FQ_F8_MX:
        got = scales.cpu().numpy().astype(np.int64)
        lo, hi = oracle.mx8_scale_code(amax * (1 - 64 * U)), oracle.mx8_scale_code(amax * (1 + 64 * U))
        assert np.all((got >= lo) & (got <= hi))
        s = 2.0 ** (got - 127.0)
    else:
        s = f64(scales).reshape(rows, 1)
        assert np.all(np.abs(s - amax / 448) <= 66 * U * amax / 448 + 2.0 ** -126)
    s = np.repeat(s, width, 1)
    v = oracle.float8_decode(codes, oracle.E4M3) * s
    assert np.all(np.abs(v - n) <= np.maximum(2.0 ** -4 * np.abs(n), 2.0 ** -10 * s) + 70 * U * np.abs(n))
    return v


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("stream", ["none", "bf16", "f32"])
def test_forward(cols, stream):
    for rows in (1, 2, 5, 19):
        x, res, gamma, h = inputs(rows, cols, stream, seed=rows)
        rstd = torch.full((rows,), 7.0, device=DEV)
        hg, y = fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, rstd=rstd)
        n, r = oracle.rmsnorm(h, f64(gamma), EPS)
        if res is None:
            assert hg is None
        else:
            assert np.array_equal(f64(hg), h.astype(np.float64))
        assert np.all(np.abs(f64(rstd) - r) <= 64 * U * r)
        assert np.all(np.abs(f64(y) - n) <= (2.0 ** -8 + 64 * U) * np.abs(n)), (rows, cols)


@pytest.mark.parametrize("cols", [32, 96, 512, 544, 1056, 2080, 2880, 4096, 4128, 8224, 16416, 32768])
@pytest.mark.parametrize("f8", [fq.FQ_F8_MX, fq.FQ_F8_ROW])
@pytest.mark.parametrize("stream", ["none", "bf16", "f32"])
def test_forward_8bit(cols, f8, stream):
    for rows in (1, 6):
        x, res, gamma, h = inputs(rows, cols, stream, seed=cols, gamma_type=torch.bfloat16)
        n, _ = oracle.rmsnorm(h, f64(gamma), EPS)
        _, codes, scales = fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, f8=f8)
        v = check_codes(n, codes, scales, f8, cols)
        # with y the same codes and the values they stand for
        y = torch.empty_like(x)
        _, codes2, scales2 = fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, f8=f8, y=y)
        assert torch.equal(codes, codes2) and torch.equal(scales, scales2)
        if f8 == fq.FQ_F8_MX:
            assert np.array_equal(f64(y), v)
        else:
            assert np.all(np.abs(f64(y) - v) <= (2.0 ** -8 + U) * np.abs(v))


def test_forward_8bit_y_alone():
    """Through the C entry: y without codes and scales."""
    x, _, gamma, h = inputs(3, 64, "none")
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    fq.fq_rmsnorm_fwd(x, gamma, EPS, f8=fq.FQ_F8_MX, y=y)
    st = fq.lib().fq_rmsnorm_fwd(x.data_ptr(), None, 0, gamma.data_ptr(), 1, EPS, 3, 64, 1, None,
                                 y2.data_ptr(), None, None, None, torch.cuda.current_stream().cuda_stream)
    assert st == fq.FQ_OK
    assert torch.equal(y, y2)


@pytest.mark.parametrize("f8", [fq.FQ_F8_NONE, fq.FQ_F8_MX, fq.FQ_F8_ROW])
def test_rows_with_infinities_nan_and_zeros(f8):
    rows, cols = 7, 128
    x, _, gamma, h = inputs(rows, cols, "none", seed=3)
    x[1, 5] = float("nan")
    x[2, 40] = float("inf")
    x[3] = 0
    x[4] = -0.0
    x[5, :64] = 0
    y = torch.empty_like(x)
    out = fq.fq_rmsnorm_fwd(x, gamma, 0.0 if f8 == fq.FQ_F8_NONE else EPS, f8=f8, y=y)
    y = y.float().cpu()
    # a NaN reaches the row's statistic; an infinity makes it infinite, so r is 0:
    # NaN at the infinity (and what shares its scale), 0 elsewhere
    assert torch.isnan(y[1]).all()
    width = {fq.FQ_F8_NONE: 1, fq.FQ_F8_MX: 32, fq.FQ_F8_ROW: cols}[f8]
    hit = torch.arange(cols) // width == 40 // width
    assert torch.isnan(y[2, hit]).all() and (y[2, ~hit] == 0).all()
    if f8 == fq.FQ_F8_NONE:
        assert torch.isnan(y[3]).all()           # 0 / sqrt(0)
    else:
        assert (y[3] == 0).all() and (y[4] == 0).all()
        codes, scales = out[1].cpu(), out[2].cpu()
        assert (codes[1] == 0x7F).all() and (codes[2, hit] == 0x7F).all()
        if f8 == fq.FQ_F8_MX:
            assert (scales[1] == 255).all() and scales[2, 1] == 255 and (scales[3] == 0).all()
            assert (scales[5, :2] == 0).all() and (codes[5, :64] == 0).all()
        else:
            assert torch.isnan(scales[1:3]).all() and scales[3] == 2.0 ** -126
    fine = y[[0, 5, 6]]
    assert torch.isfinite(fine).all()
    n, _ = oracle.rmsnorm(f64(x)[[0, 6]], f64(gamma), 0.0 if f8 == fq.FQ_F8_NONE else EPS)
    half = {fq.FQ_F8_NONE: 2.0 ** -8}.get(f8, 2.0 ** -4 + 2.0 ** -8)
    assert np.all(np.abs(y[[0, 6]].double().numpy() - n) <= half * np.abs(n) * 1.001 + (0 if f8 == 0 else 2.0 ** -10 * np.abs(n).max() / 200))


def test_in_place_stream():
    x, res, gamma, h = inputs(33, 2880, "bf16")
    want = fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res)
    got = fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, h=res)
    assert got[0] is res and torch.equal(want[0], res) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("stream", ["none", "bf16", "f32"])
def test_backward(cols, stream):
    for rows in (1, 3, 70) if cols < 20000 else (1, 5):
        x, res, gamma, h = inputs(rows, cols, stream, seed=rows)
        rng = np.random.default_rng(9)
        hg = torch.tensor(h, device=DEV).to(torch.float32 if stream == "f32" else torch.bfloat16)
        _, r = oracle.rmsnorm(h, f64(gamma), EPS)
        rstd = torch.tensor(r, dtype=torch.float32, device=DEV)
        dy = bf(rng.standard_normal((rows, cols)) * 1e-3).to(DEV)
        dres = None if stream == "none" else bf(rng.standard_normal((rows, cols)) * 1e-3).to(DEV).to(hg.dtype)
        dx = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV) if stream == "f32" else None
        dh, dgamma = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, dres=dres, dx=dx)
        r32 = f64(rstd)
        want, wg = oracle.rmsnorm_bwd(f64(dy), h, f64(gamma), r32, None if dres is None else f64(dres))
        xh, g = h * r32[:, None], f64(dy) * f64(gamma)
        size = r32[:, None] * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
        fp32 = 80 * U * size + 2 * U * np.abs(want)
        half = U if stream == "f32" else 2.0 ** -8
        assert np.all(np.abs(f64(dh) - want) <= half * np.abs(want) + (1 + half) * fp32), (rows, cols)
        if dx is not None:
            assert torch.equal(dx, dh.to(torch.bfloat16))
        assert np.all(np.abs(f64(dgamma) - wg) <= (rows + 8) * U * np.abs(f64(dy) * xh).sum(0) + 1e-30)


def test_backward_many_rows_is_repeatable_and_in_place():
    rows, cols = 4099, 1000
    x, res, gamma, h = inputs(rows, cols, "bf16")
    hg = torch.tensor(h, device=DEV).to(torch.bfloat16)
    rstd = torch.tensor(oracle.rmsnorm(h, f64(gamma), EPS)[1], dtype=torch.float32, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    dy = torch.randn((rows, cols), device=DEV, generator=g).to(torch.bfloat16)
    dres = torch.randn((rows, cols), device=DEV, generator=g).to(torch.bfloat16)
    a = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, dres=dres)
    ws = fq.rmsnorm_bwd_workspace(rows, cols, DEV)
    ws.fill_(0xFF)                                   # what the workspace held does not matter
    b = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, dres=dres, ws=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c, none = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd, dres=dres, dh=dres, need_dgamma=False)
    assert none is None and c is dres and torch.equal(a[0], dres)
    _, wg = oracle.rmsnorm_bwd(f64(dy), h, f64(gamma), f64(rstd))
    xh = h * f64(rstd)[:, None]
    assert np.all(np.abs(f64(a[1]) - wg) <= (rows + 8) * U * np.abs(f64(dy) * xh).sum(0))


def test_forward_then_backward_is_the_gradient():
    """The device's own forward and backward against differences of the float64
    forward at the same point (FP32 stream, so the point is exact)."""
    rows, cols = 2, 33
    x, res, gamma, h = inputs(rows, cols, "f32", seed=8)
    rstd = torch.empty(rows, device=DEV)
    hg, _ = fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, rstd=rstd)
    dy = bf(np.random.default_rng(2).standard_normal((rows, cols))).to(DEV)
    dh, dgamma = fq.fq_rmsnorm_bwd(dy, hg, gamma, rstd)
    h64, g64, d64 = f64(hg), f64(gamma), f64(dy)
    d = 1e-5
    for i in np.ndindex(h64.shape):
        e = np.zeros_like(h64)
        e[i] = d
        diff = ((oracle.rmsnorm(h64 + e, g64, EPS)[0] - oracle.rmsnorm(h64 - e, g64, EPS)[0]) * d64).sum() / (2 * d)
        assert abs(diff - f64(dh)[i]) <= 1e-5
    for c in range(cols):
        e = np.zeros(cols)
        e[c] = d
        diff = ((oracle.rmsnorm(h64, g64 + e, EPS)[0] - oracle.rmsnorm(h64, g64 - e, EPS)[0]) * d64).sum() / (2 * d)
        assert abs(diff - f64(dgamma)[c]) <= 1e-5


def test_another_stream_and_graph_replays():
    rows, cols = 300, 2880
    x, res, gamma, _ = inputs(rows, cols, "bf16")
    rstd, h, y = torch.empty(rows, device=DEV), torch.empty_like(res), torch.empty_like(x)
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=DEV)
    dh, dgamma = torch.empty_like(res), torch.empty(cols, device=DEV)
    ws = fq.rmsnorm_bwd_workspace(rows, cols, DEV)
    outs = [rstd, h, y, codes, scales, dh, dgamma]

    def both(stream=None):
        fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, f8=fq.FQ_F8_MX, h=h, y=y, codes=codes, scales=scales,
                          rstd=rstd, stream=stream)
        fq.fq_rmsnorm_bwd(y, h, gamma, rstd, dres=res, dh=dh, dgamma=dgamma, ws=ws, stream=stream)

    both()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        both()
    for _ in range(3):
        for t in outs:
            t.zero_()
        fq.fq_rmsnorm_fwd(x[:5].contiguous(), gamma, EPS)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_beyond_32_bit_offsets():
    """More than 2^32 elements: first and last rows against float64."""
    cols = 32768
    rows = (1 << 32) // cols + 3
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    x.fill_(0.5)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    for r in (0, rows - 1):
        x[r] = torch.randn(cols, generator=gen, device=DEV)
    gamma = torch.ones(cols, device=DEV)
    y = torch.empty_like(x)
    rstd = torch.empty(rows, device=DEV)
    fq.fq_rmsnorm_fwd(x, gamma, EPS, y=y, rstd=rstd)
    for r in (0, rows - 1):
        n, _ = oracle.rmsnorm(f64(x[r: r + 1]), np.ones(cols), EPS)
        assert np.all(np.abs(f64(y[r: r + 1]) - n) <= (2.0 ** -8 + 64 * U) * np.abs(n))
    last = x[-1:].clone()
    dh = y
    fq.fq_rmsnorm_bwd(x, x, gamma, rstd, dh=dh, need_dgamma=False)
    want, _ = oracle.rmsnorm_bwd(f64(last), f64(last), np.ones(cols), f64(rstd[-1:]))
    xh = f64(last) * f64(rstd[-1:])
    size = f64(rstd[-1:]) * (np.abs(f64(last)) + np.abs(xh) * np.abs(f64(last) * xh).mean())
    assert np.all(np.abs(f64(dh[-1:]) - want) <= 2.0 ** -8 * np.abs(want) + 82 * U * size)
