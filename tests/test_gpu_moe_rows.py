"""Expert sorting and its row operators over every width class and over more
tokens than one group, one launch or one grid takes.  Error bounds as in
test_gpu_moe: (k + 2) 2^-24 of the sum of magnitudes and 2^-8 of a BF16 value
for combine, (cols + 2) 2^-24 of the sum of magnitudes for a weight's gradient."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import step as oracle
from test_gpu_moe import U, f64, make_ids, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T, k", [(2047, 1), (2048, 1), (2051, 1), (2050, 2), (2049, 2), (2049, 3), (500, 5), (5, 2), (1, 1)])
@pytest.mark.parametrize("H", [8, 64, 72, 128, 136, 256, 264, 512, 520, 2880, 4096, 4104])
def test_widths(T, k, H):
    E, align = 7, 16
    ids = make_ids(T, k, E, "masked", seed=T + H)
    q = fq.fq_moe_sort(torch.tensor(ids, device=DEV), E, align)
    rows = q.src.numel()
    _, pos, src = oracle.moe_sort(ids, E, align, rows)
    assert np.array_equal(q.pos.cpu().numpy(), pos) and np.array_equal(q.src.cpu().numpy(), src)
    x, y, dout = normal((T, H), 1), normal((rows, H), 2), normal((T, H), 3, 1e-3)
    w = torch.tensor(np.random.default_rng(3).random((T, k)), dtype=torch.float32, device=DEV)
    out = torch.full((rows, H), 9.0, dtype=torch.bfloat16, device=DEV)
    fq.fq_moe_dispatch(x, q, y=out)
    assert np.array_equal(f64(out), oracle.moe_rows_of(f64(x), src, k))
    got = np.where((pos >= 0)[..., None], f64(y)[np.maximum(pos, 0)], 0.0)           # [T, k, H]
    for weights in (w, None):
        scale = np.ones((T, k)) if weights is None else f64(w)
        want, size = (got * scale[..., None]).sum(1), (np.abs(got) * scale[..., None]).sum(1)
        c = fq.fq_moe_combine(y, q, weights)
        assert np.all(np.abs(f64(c) - want) <= 2.0 ** -8 * np.abs(want) + (k + 2) * U * size)
    dy = torch.full((rows, H), 9.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((T, k), 9.0, device=DEV)
    fq.fq_moe_combine_bwd(dout, y, q, w, dy=dy, dweights=dw)
    a = np.maximum(src, 0)
    wdy = np.where((src >= 0)[:, None], f64(dout)[a // k] * f64(w).reshape(-1)[a][:, None], 0.0)
    assert np.all(np.abs(f64(dy) - wdy) <= (2.0 ** -8 + 2 * U) * np.abs(wdy))
    wdw, size = (got * f64(dout)[:, None]).sum(2), (np.abs(got) * np.abs(f64(dout))[:, None]).sum(2)
    assert np.all(np.abs(f64(dw) - wdw) <= (H + 2) * U * size)


@pytest.mark.parametrize("n", [1, 63, 1023, 1024, 1025, 2048, 8191, 8192, 8193, 262144, 262145, 300007])
@pytest.mark.parametrize("E", [1, 3, 256, 1024])
def test_sort_lengths(n, E):
    """Around a step, the lengths that every workgroup counts whole, and the most
    workgroups."""
    ids = make_ids(n, 1, E, "masked", seed=n)
    rows = fq.moe_rows(n, 1, E, 8)
    q = fq.fq_moe_sort(torch.tensor(ids, device=DEV), E, 8)
    offsets, pos, src = oracle.moe_sort(ids, E, 8, rows)
    assert np.array_equal(q.offsets.cpu().numpy(), offsets)
    assert np.array_equal(q.pos.cpu().numpy(), pos)
    assert np.array_equal(q.src.cpu().numpy(), src)


def test_more_tokens_than_a_grid_takes():
    T, H = (1 << 27) + (1 << 20) + 5, 8
    ids = (torch.arange(T, dtype=torch.int32, device=DEV) % 3).view(T, 1) - 1      # a third without an expert
    q = fq.fq_moe_sort(ids, 2, 1)
    used = int(q.offsets[2])
    assert used == int((ids >= 0).sum()) and int(q.offsets[1]) == int((ids == 0).sum())
    assert torch.equal(q.pos.view(-1) < 0, ids.view(-1) < 0)
    assert torch.equal(q.src[q.pos[ids >= 0].long()], torch.arange(T, dtype=torch.int32, device=DEV)[ids.view(-1) >= 0])
    assert (q.src[:used].diff()[torch.arange(used - 1, device=DEV) != int(q.offsets[1]) - 1] == 3).all()
    assert (q.src[used:] == -1).all()
    x = (torch.arange(T, device=DEV) % 251).to(torch.bfloat16)[:, None].expand(T, H).contiguous()
    y = fq.fq_moe_dispatch(x, q)
    # the rows' expected values from src itself, a part at a time (indexing x with
    # all of src at once gives wrong rows at this size)
    for a in range(0, used, 1 << 22):
        src = q.src[a: min(used, a + (1 << 22))]
        assert torch.equal(y[a: a + src.numel()], (src % 251).to(torch.bfloat16)[:, None].expand(-1, H))
    assert (y[used:] == 0).all()
    w = torch.full((T, 1), 2.0, device=DEV)
    out = fq.fq_moe_combine(y, q, w)
    assert torch.equal(out, torch.where(ids >= 0, 2 * x, torch.zeros_like(x)))
    dy, dw = fq.fq_moe_combine_bwd(x, y, q, w)
    assert torch.equal(dy, 2 * y)
    assert torch.equal(dw, torch.where(ids >= 0, (x.float() ** 2).sum(1, keepdim=True), torch.zeros_like(w)))


@pytest.mark.parametrize("k", [3, 4, 5, 6, 7, 8, 9, 13, 16, 17, 64])
@pytest.mark.parametrize("T", [1, 37, 513])
@pytest.mark.parametrize("H", [64, 136, 512, 1056])
def test_assignments_of_a_token(T, k, H):
    test_widths(T, k, H)
