"""Tokens sorted by expert, dispatch, combine and their backward on the GPU.
The sort and the dispatch are exact; combine sums k products in FP32 (error at
most (k + 1) 2^-24 of the sum of magnitudes) and rounds to BF16 (2^-8 of the
value); a weight's gradient is a sum of cols products (cols 2^-24 of the sum of
magnitudes, whatever the order)."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import step as oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


def make_ids(T, k, E, kind, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "one":                               # every token to the same experts
        return np.tile((np.arange(k) * 7) % E, (T, 1)).astype(np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)      # a token may name an expert twice
    if kind == "masked":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.05] = E + 3             # no such expert
        ids[rng.random((T, k)) < 0.02] = -2 ** 31
        ids[rng.random(T) < 0.2] = -1
    return ids


def normal(shape, seed, sigma=1.0):
    return (torch.tensor(np.random.default_rng(seed).standard_normal(shape), dtype=torch.float32)
            * sigma).to(torch.bfloat16).to(DEV)


SORTS = [(1, 1, 1, 1), (1, 4, 32, 1), (3, 2, 5, 16), (64, 1, 2, 128), (63, 3, 1024, 1), (700, 4, 32, 64),
         (2047, 1, 7, 3), (2049, 1, 7, 128), (1021, 8, 128, 64), (5000, 6, 1000, 100), (70001, 4, 33, 1024),
         (3, 64, 64, 8)]


@pytest.mark.parametrize("T, k, E, align", SORTS)
@pytest.mark.parametrize("kind", ["random", "masked", "one", "none"])
def test_sort(T, k, E, align, kind):
    ids = make_ids(T, k, E, kind, seed=T)
    rows = fq.moe_rows(T, k, E, align)
    q = fq.MoeSorted(torch.full((E + 1,), 77, dtype=torch.int32, device=DEV),
                     torch.full((T, k), 77, dtype=torch.int32, device=DEV),
                     torch.full((rows,), 77, dtype=torch.int32, device=DEV))
    ws = fq.moe_sort_workspace(T, k, E, DEV)
    ws.fill_(0xFF)
    fq.fq_moe_sort(torch.tensor(ids, device=DEV), E, align, out=q, ws=ws)
    offsets, pos, src = oracle.moe_sort(ids, E, align, rows)
    assert np.array_equal(q.offsets.cpu().numpy(), offsets)
    assert np.array_equal(q.pos.cpu().numpy(), pos)
    assert np.array_equal(q.src.cpu().numpy(), src)


def test_sort_more_rows_than_needed():
    ids = make_ids(100, 2, 4, "random")
    rows = fq.moe_rows(100, 2, 4, 32) + 1000
    q = fq.MoeSorted(torch.empty(5, dtype=torch.int32, device=DEV), torch.empty((100, 2), dtype=torch.int32, device=DEV),
                     torch.zeros(rows, dtype=torch.int32, device=DEV))
    fq.fq_moe_sort(torch.tensor(ids, device=DEV), 4, 32, out=q)
    assert np.array_equal(q.src.cpu().numpy(), oracle.moe_sort(ids, 4, 32, rows)[2])


ROWS = [(1, 4, 32, 1, 8), (1, 1, 1, 64, 2880), (5, 3, 4, 16, 96), (130, 4, 8, 128, 1000), (257, 8, 128, 64, 2088),
        (40, 64, 64, 1, 4128)]


@pytest.mark.parametrize("T, k, E, align, H", ROWS)
@pytest.mark.parametrize("kind", ["random", "masked", "none"])
def test_dispatch_combine_and_backward(T, k, E, align, H, kind):
    ids = make_ids(T, k, E, kind, seed=H)
    q = fq.fq_moe_sort(torch.tensor(ids, device=DEV), E, align)
    rows = q.src.numel()
    _, pos, src = oracle.moe_sort(ids, E, align, rows)
    x = normal((T, H), 1)
    rows_out = torch.full((rows, H), 9.0, dtype=torch.bfloat16, device=DEV)
    fq.fq_moe_dispatch(x, q, y=rows_out)
    assert np.array_equal(f64(rows_out), oracle.moe_rows_of(f64(x), src, k))
    y = normal((rows, H), 2)
    y[torch.tensor(src, device=DEV) < 0] = float("nan")       # padding rows are not read
    w = torch.tensor(np.random.default_rng(3).random((T, k)), dtype=torch.float32, device=DEV)
    y64 = np.nan_to_num(f64(y))
    for weights in (w, None):
        out = fq.fq_moe_combine(y, q, weights)
        want = oracle.moe_combine(y64, pos, None if weights is None else f64(w))
        size = oracle.moe_combine(np.abs(y64), pos, None if weights is None else f64(w))
        assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (k + 2) * U * size)
    dout = normal((T, H), 4, 1e-3)
    dy = torch.full((rows, H), 9.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((T, k), 9.0, device=DEV)
    fq.fq_moe_combine_bwd(dout, y, q, w, dy=dy, dweights=dw)
    wdy, wdw = oracle.moe_combine_bwd(f64(dout), y64, pos, f64(w))
    _, size = oracle.moe_combine_bwd(np.abs(f64(dout)), np.abs(y64), pos, f64(w))
    assert np.all(np.abs(f64(dy) - wdy) <= (2.0 ** -8 + 2 * U) * np.abs(wdy))
    assert np.all(np.abs(f64(dw) - wdw) <= (H + 2) * U * size)


@pytest.mark.parametrize("f8", [fq.FQ_F8_MX, fq.FQ_F8_ROW])
@pytest.mark.parametrize("T, k, E, align, H", [(1, 4, 32, 1, 32), (37, 2, 5, 16, 2880), (300, 4, 8, 64, 1056)])
def test_dispatch_of_8bit_rows(f8, T, k, E, align, H):
    """The codes and scales of the norm, decoded while they are sorted."""
    x = normal((T, H), 5)
    if T > 1:
        x[T // 2, 3] = float("inf")                            # a block, or row, that stands for NaN
    y = torch.empty_like(x)
    _, codes, scales = fq.fq_rmsnorm_fwd(x, torch.ones(H, device=DEV), 1e-5, f8=f8, y=y)
    ids = make_ids(T, k, E, "masked" if T > 1 else "random", seed=6)
    q = fq.fq_moe_sort(torch.tensor(ids, device=DEV), E, align)
    got = fq.fq_moe_dispatch(codes, q, f8=f8, scales=scales)
    src = oracle.moe_sort(ids, E, align, q.src.numel())[2]
    assert np.array_equal(f64(got), oracle.moe_rows_of(f64(y), src, k), equal_nan=True)


def test_entries_outside_the_buffers_count_as_none():
    T, k, H, rows = 6, 2, 64, 10
    pos = torch.tensor([[0, -1], [3, 10], [2 ** 31 - 1, -2 ** 31], [5, 6], [-7, 9], [1, 2]], dtype=torch.int32, device=DEV)
    src = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    ok = (pos >= 0) & (pos < rows)
    src[pos[ok].long()] = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)[ok]
    src[4], src[7] = T * k, 2 ** 31 - 1                        # no such assignments: padding
    q = fq.MoeSorted(None, pos, src)
    p = pos.cpu().numpy()
    p = np.where((p >= 0) & (p < rows), p, -1)
    s = src.cpu().numpy()
    s = np.where((s >= 0) & (s < T * k), s, -1)
    x, y, dout = normal((T, H), 1), normal((rows, H), 2), normal((T, H), 3)
    w = torch.rand((T, k), device=DEV)
    assert np.array_equal(f64(fq.fq_moe_dispatch(x, q)), oracle.moe_rows_of(f64(x), s, k))
    want = oracle.moe_combine(f64(y), p, f64(w))
    assert np.all(np.abs(f64(fq.fq_moe_combine(y, q, w)) - want) <= 2.0 ** -8 * np.abs(want) + 4 * U * 10)
    dy, dw = fq.fq_moe_combine_bwd(dout, y, q, w)
    wdy, wdw = oracle.moe_combine_bwd(f64(dout), f64(y), p, f64(w))
    assert np.all(np.abs(f64(dy) - wdy) <= (2.0 ** -8 + 2 * U) * np.abs(wdy))
    assert np.all((f64(dw) == 0) == (p < 0))


def test_infinities_and_nan_travel():
    T, k, H = 3, 2, 16
    q = fq.fq_moe_sort(torch.tensor([[0, 1], [1, 0], [-1, 1]], dtype=torch.int32, device=DEV), 2, 4)
    y = normal((q.src.numel(), H), 1)
    r = q.pos[0, 0]
    y[r, 3], y[r, 4] = float("inf"), float("nan")
    w = torch.full((T, k), 0.5, device=DEV)
    out = fq.fq_moe_combine(y, q, w).float().cpu()
    assert torch.isinf(out[0, 3]) and torch.isnan(out[0, 4])
    assert torch.isfinite(out[1:]).all() and torch.isfinite(out[0, 5:]).all()


def test_graph_replays_and_another_stream():
    T, k, E, align, H = 600, 4, 16, 64, 512
    ids = torch.tensor(make_ids(T, k, E, "masked"), device=DEV)
    x, w = normal((T, H), 1), torch.rand((T, k), device=DEV)
    rows = fq.moe_rows(T, k, E, align)
    i32 = dict(dtype=torch.int32, device=DEV)
    q = fq.MoeSorted(torch.empty(E + 1, **i32), torch.empty((T, k), **i32), torch.empty(rows, **i32))
    ws = fq.moe_sort_workspace(T, k, E, DEV)
    y, out = torch.empty((rows, H), dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    outs = [q.offsets, q.pos, q.src, y, out, dy, dw]

    def step(stream=None):
        fq.fq_moe_sort(ids, E, align, out=q, ws=ws, stream=stream)
        fq.fq_moe_dispatch(x, q, y=y, stream=stream)
        fq.fq_moe_combine(y, q, w, out=out, stream=stream)
        fq.fq_moe_combine_bwd(x, y, q, w, dy=dy, dweights=dw, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        step()
    for _ in range(3):
        for t in outs:
            t.zero_()
        fq.fq_moe_combine(dy, q, None)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_beyond_32_bit_offsets():
    """Row offsets past 2^32 elements, at both ends of the buffers."""
    H, T, k = 65536, 65540, 1
    rows = T
    i32 = dict(dtype=torch.int32, device=DEV)
    q = fq.fq_moe_sort(torch.zeros((T, k), **i32), 1, 1)
    assert q.src.numel() == rows
    x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    x.copy_(torch.arange(T, device=DEV, dtype=torch.float32)[:, None].remainder(251).expand(T, H))
    y = fq.fq_moe_dispatch(x, q)
    assert torch.equal(y[-1], x[-1]) and torch.equal(y[0], x[0]) and torch.equal(y[65537], x[65537])
    w = torch.full((T, k), 2.0, device=DEV)
    out = fq.fq_moe_combine(y, q, w, out=x)
    assert torch.equal(out[-1].float(), 2 * y[-1].float())
    dy, dw = fq.fq_moe_combine_bwd(out, y, q, w, dy=out)
    assert torch.equal(dy[-1].float(), 4 * y[-1].float())
    v = float((T - 1) % 251)
    assert float(dw[-1, 0]) == pytest.approx(2 * v * v * H, rel=1e-3)
