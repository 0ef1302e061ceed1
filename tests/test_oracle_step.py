"""Pins of the oracle of the operators around the linears: 8-bit formats
against torch's types, gradients against differences of the forward, the sort
against its properties, stochastic rounding against its mean."""
import numpy as np
import pytest
import torch

from oracle import step


@pytest.mark.parametrize("table, dtype", [(step.E4M3, torch.float8_e4m3fn), (step.E5M2, torch.float8_e5m2)])
def test_float8_tables_are_torchs(table, dtype):
    want = torch.arange(128, dtype=torch.uint8).view(dtype).float().numpy()
    assert np.array_equal(table.astype(np.float32), want, equal_nan=True)


@pytest.mark.parametrize("table", [step.E4M3, step.E5M2])
def test_float8_sr_is_unbiased_and_exact_on_the_grid(table):
    finite = table[np.isfinite(table)]
    r = np.arange(65536)
    for a in (finite[3], finite[40], finite[-1]):
        assert np.all(float(a) == table[step.float8_sr(np.full(r.size, a), r, table)])
    for k in (0, 2, 9, 70, finite.size - 2):
        a = finite[k] + 0.3125 * (finite[k + 1] - finite[k])       # 0.3125 * 2^16 is whole
        got = table[step.float8_sr(np.full(r.size, a), r, table)]
        assert set(got) == {finite[k], finite[k + 1]}
        assert got.mean() == pytest.approx(a, rel=1e-12)


def test_mx8_scale_never_saturates_and_is_the_smallest():
    amax = np.array([1.0, 448.0, 448.0 * (1 + 2 ** -23), 449.0, 512.0, 1.75, 1.7500001, 3e38, 1e-30])
    s = 2.0 ** (step.mx8_scale_code(amax) - 127)
    assert np.all(amax <= 448 * s) and np.all(amax > 448 * s / 2)
    assert step.mx8_scale_code(np.array([0.0]))[0] == 0


def test_norm_backward_against_differences():
    rng = np.random.default_rng(0)
    x, res, dy, dres = (rng.standard_normal((3, 7)) for _ in range(4))
    gamma, eps = 1 + 0.3 * rng.standard_normal(7), 1e-3

    def loss(h, gam):
        return (step.rmsnorm(h, gam, eps)[0] * dy).sum() + (h * dres).sum()

    h = x + res
    dh, dgamma = step.rmsnorm_bwd(dy, h, gamma, step.rmsnorm(h, gamma, eps)[1], dres)
    d = 1e-6
    for i in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[i] = d
        assert (loss(h + e, gamma) - loss(h - e, gamma)) / (2 * d) == pytest.approx(dh[i], abs=1e-7)
    for c in range(7):
        e = np.zeros(7)
        e[c] = d
        assert (loss(h, gamma + e) - loss(h, gamma - e)) / (2 * d) == pytest.approx(dgamma[c], abs=1e-7)


def test_combine_backward_against_differences():
    rng = np.random.default_rng(1)
    ids = np.array([[0, 2], [1, -1], [2, 2], [-1, -1]], np.int32)
    _, pos, src = step.moe_sort(ids, 3, 4, 12)
    y, w, dout = rng.standard_normal((12, 5)), rng.standard_normal((4, 2)), rng.standard_normal((4, 5))
    dy, dw = step.moe_combine_bwd(dout, y, pos, w)
    f = lambda y, w: (step.moe_combine(y, pos, w) * dout).sum()  # noqa: E731
    d = 1e-6
    for i in np.ndindex(y.shape):
        e = np.zeros_like(y)
        e[i] = d
        assert (f(y + e, w) - f(y - e, w)) / (2 * d) == pytest.approx(dy[i], abs=1e-8)
    for i in np.ndindex(w.shape):
        e = np.zeros_like(w)
        e[i] = d
        assert (f(y, w + e) - f(y, w - e)) / (2 * d) == pytest.approx(dw[i], abs=1e-8)
    # dispatch and the unweighted combine are each other's transpose
    x = rng.standard_normal((4, 5))
    assert (step.moe_rows_of(x, src, 2) * y).sum() == pytest.approx((x * step.moe_combine(y, pos)).sum())


def test_sort_is_stable_and_padded():
    rng = np.random.default_rng(2)
    ids = rng.integers(-1, 6, (40, 3)).astype(np.int32)
    offsets, pos, src = step.moe_sort(ids, 5, 8, 200)
    assert np.all(offsets % 8 == 0) and offsets[0] == 0
    flat = ids.reshape(-1)
    live = (flat >= 0) & (flat < 5)
    assert np.array_equal(pos.reshape(-1) >= 0, live)
    assert np.array_equal(src[pos.reshape(-1)[live]], np.flatnonzero(live))
    for e in range(5):
        seg = src[offsets[e]: offsets[e + 1]]
        seg = seg[seg >= 0]
        assert np.all(np.diff(seg) > 0) and np.all(flat[seg] == e)


def test_adamw_is_torchs():
    rng = np.random.default_rng(3)
    w0 = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.tensor(w0, dtype=torch.float64))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
    w, m, v = w0, np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.tensor(2 * g)
        opt.step()
        w, m, v = step.adamw(w, g, m, v, lr=1e-2, step=t, beta1=0.9, beta2=0.95, eps=1e-6,
                             weight_decay=0.1, scale=2.0)
    assert np.allclose(p.detach().numpy(), w, rtol=1e-12, atol=0)


def test_a_stochastic_second_moment_follows_the_gradient():
    """Rounded to nearest, an 8-bit v at beta2 = 0.999 would stay where it is;
    rounded stochastically it follows a gradient that grows ten times."""
    n = 128
    v = np.full(n, 1e-6, np.float32)
    rng = np.random.default_rng(4)
    for t in range(1500):
        v = np.float32(0.999) * v + np.float32(0.001) * np.float32(1e-4)
        codes, s = step.quantize_state(v, rng.integers(0, 65536, n), step.E5M2_MAX, step.E5M2, True)
        v = (step.float8_decode(codes, step.E5M2) * s[0]).astype(np.float32)
    want = 1e-4 - (1e-4 - 1e-6) * 0.999 ** 1500
    assert abs(v.mean() / want - 1) < 0.15
