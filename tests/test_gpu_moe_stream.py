"""Dispatch, combine and its backward in calls that stream (from 2^25 elements of
assigned rows on, the backward from 2^24), in every class of widths and of k, and
just below: against float64 on the device.  Error bounds as in test_gpu_moe."""
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from test_gpu_moe import U

pytestmark = pytest.mark.gpu

E, ALIGN = 13, 16
SHAPES = [(525000, 1, 64), (262200, 2, 64), (131100, 4, 64), (40000, 7, 120), (32800, 8, 136), (33000, 4, 256), (16400, 4, 512),
          (9000, 9, 416), (8200, 1, 4104), (4096, 2, 4104), (4099, 3, 2736), (2913, 4, 2880), (2200, 6, 2880), (1500, 8, 2880),
          (8185, 1, 4096), (2047, 4, 4096)]


def inputs(T, k, H):
    g = torch.Generator(device=DEV)
    g.manual_seed(T + H)
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    ids[torch.rand((T, k), generator=g, device=DEV) < 0.1] = -1
    ids[torch.rand(T, generator=g, device=DEV) < 0.05] = -1
    q = fq.fq_moe_sort(ids, E, ALIGN)
    live = q.pos.view(-1) >= 0
    assert torch.equal(live, ids.view(-1) >= 0)
    assert torch.equal(q.src[q.pos.view(-1)[live].long()], torch.arange(T * k, device=DEV, dtype=torch.int32)[live])
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    return g, q, normal


def filled(rows, H):
    return torch.full((rows, H), 9.0, dtype=torch.bfloat16, device=DEV)


def by_row(values, q, k):
    """Row src // k of values for every row that has an assignment, 0 elsewhere."""
    a = q.src.clamp_min(0).long() // k
    return torch.where((q.src >= 0)[:, None], values[a], torch.zeros((), dtype=values.dtype, device=DEV))


@pytest.mark.parametrize("T, k, H", SHAPES)
def test_bf16_rows(T, k, H):
    g, q, normal = inputs(T, k, H)
    rows = q.src.numel()
    x, y = normal(T, H), normal(rows, H)
    assert torch.equal(fq.fq_moe_dispatch(x, q, y=filled(rows, H)), by_row(x, q, k))
    y[q.src < 0] = float("nan")                                  # padding rows are not read
    w = torch.rand((T, k), generator=g, device=DEV)
    dout = (normal(T, H).float() * 1e-3).to(torch.bfloat16)
    dy = filled(rows, H)
    dw = torch.full((T, k), 9.0, device=DEV)
    fq.fq_moe_combine_bwd(dout, y, q, w, dy=dy, dweights=dw)
    for weights in (w, None):
        out = fq.fq_moe_combine(y, q, weights, out=filled(T, H))
        want, size = (torch.zeros((T, H), dtype=torch.float64, device=DEV) for _ in range(2))
        for j in range(k):
            live = q.pos[:, j] >= 0
            v = torch.where(live[:, None], y[q.pos[:, j].clamp_min(0).long()].double(), 0.0)
            v = v if weights is None else v * w[:, j, None].double()
            want += v
            size += v.abs()
        assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (k + 2) * U * size).all()
    wdy = by_row(dout, q, k).double() * w.view(-1)[q.src.clamp_min(0).long()][:, None].double()
    assert ((dy.double() - wdy).abs() <= (2.0 ** -8 + 2 * U) * wdy.abs()).all()
    for j in range(k):
        live = q.pos[:, j] >= 0
        v = torch.where(live[:, None], y[q.pos[:, j].clamp_min(0).long()].double(), 0.0) * dout.double()
        assert ((dw[:, j].double() - v.sum(1)).abs() <= (H + 2) * U * v.abs().sum(1)).all()
        assert (dw[~live, j] == 0).all()


@pytest.mark.parametrize("T, k, H", [(131100, 4, 64), (32800, 8, 128), (33000, 4, 256), (16400, 4, 512), (8200, 1, 4128),
                                     (4096, 2, 4128), (2913, 4, 2880), (1500, 8, 2880), (2047, 4, 4096)])
@pytest.mark.parametrize("f8", [fq.FQ_F8_MX, fq.FQ_F8_ROW])
def test_8bit_rows(T, k, H, f8):
    _, q, normal = inputs(T, k, H)
    x = normal(T, H)
    x[T // 2, 3] = float("inf")                                  # a block, or row, that stands for NaN
    _, codes, scales = fq.fq_rmsnorm_fwd(x, torch.ones(H, device=DEV), 1e-5, f8=f8)
    v = codes.view(torch.float8_e4m3fn).float()
    if f8 == fq.FQ_F8_MX:
        s = torch.ldexp(torch.ones((), device=DEV), scales.int() - 127)
        v = (v.view(T, -1, 32) * torch.where(scales == 255, float("nan"), s)[:, :, None]).view(T, H)
    else:
        v = v * scales[:, None]
    got = fq.fq_moe_dispatch(codes, q, f8=f8, scales=scales, y=filled(q.src.numel(), H))
    want = by_row(v.to(torch.bfloat16), q, k)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(got).any() == (q.pos[T // 2] >= 0).any()
    assert torch.equal(got.nan_to_num(5.0), want.nan_to_num(5.0))
