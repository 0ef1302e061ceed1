"""Calls of the feed-forward products: what the binding refuses beside what the
library does, other streams, captured graphs, and a training step's run of them
with the norm and the expert sort around them."""
import math

import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import products as op
from product_util import normal, offsets_of

pytestmark = pytest.mark.gpu


def refused(call, match):
    with pytest.raises(ValueError, match=match):
        call()


def test_refusals():
    x, w, o = normal(0, 6, 64), normal(1, 64, 96), offsets_of([0, 2, 6])
    w2 = normal(2, 2, 64, 96)
    refused(lambda: fq.fq_linear_fwd(x, w.T), "rows")
    refused(lambda: fq.fq_linear_fwd(x, normal(1, 96, 64).T), "contiguous")
    refused(lambda: fq.fq_linear_fwd(x.cpu(), w, y=normal(0, 6, 96)), "GPU")
    refused(lambda: fq.fq_linear_fwd(x.float(), w), "bfloat16")
    refused(lambda: fq.fq_linear_fwd(x, w, y=normal(0, 5, 96)), "576 are needed")
    refused(lambda: fq.fq_linear_fwd(x, w, y=torch.empty((6, 96), dtype=torch.float16, device=DEV)), "float32")
    refused(lambda: fq.fq_linear_fwd(x, w, res=normal(0, 6, 96), y=torch.empty((6, 96), device=DEV)), "float32")
    refused(lambda: fq.fq_linear_fwd(x, w, bias=normal(0, 95)), "96 are needed")
    refused(lambda: fq.fq_linear_fwd(x, w, offsets=o), "experts")
    refused(lambda: fq.fq_linear_fwd(x, w2), "w must be")
    refused(lambda: fq.fq_linear_fwd(x, w2, offsets=o.long()), "int32")
    refused(lambda: fq.fq_linear_fwd(x, w2, offsets=offsets_of([0, 2, 4, 6])), "3 are needed")
    refused(lambda: fq.fq_linear_fwd(x, w2, offsets=offsets_of([0, 6])), "3 are needed")
    refused(lambda: fq.fq_linear_fwd(x, w, pre=torch.empty((6, 96), dtype=torch.uint8, device=DEV)), "bfloat16")
    refused(lambda: fq.fq_glu_fwd(x, normal(1, 64, 97)), "even")
    refused(lambda: fq.fq_glu_bwd(normal(0, 6, 40), x, w, normal(3, 6, 96)), "rows and w's columns")
    refused(lambda: fq.fq_linear_bwd(normal(0, 5, 96), x, w), "rows and w's columns")
    refused(lambda: fq.fq_linear_bwd(normal(0, 6, 96), x, w, dw=normal(0, 64, 95)), "6144 are needed")
    with pytest.raises(TypeError):
        fq.fq_glu_fwd(x, w, bias=[0.0] * 96)
    with pytest.raises(fq.FqError) as e:
        fq.fq_linear_fwd(normal(0, 6, 60), normal(1, 60, 96))
    assert e.value.status == fq.FQ_ERR_SHAPE
    with pytest.raises(fq.FqError) as e:
        fq.fq_linear_fwd(normal(0, 1000)[1:385].view(6, 64), w)
    assert e.value.status == fq.FQ_ERR_ALIGN
    with pytest.raises(fq.FqError) as e:
        fq.fq_glu_fwd(x, w, act=fq.FQ_ACT_GELU, alpha=2.0)
    assert e.value.status == fq.FQ_ERR_DESC
    with pytest.raises(fq.FqError) as e:
        fq.fq_linear_bwd(normal(0, 6, 96), x, w, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == fq.FQ_ERR_WORKSPACE
    with pytest.raises(fq.FqError) as e:
        fq.fq_linear_bwd(normal(0, 6, 96), x, w, act=fq.FQ_ACT_SILU)
    assert e.value.status == fq.FQ_ERR_NULL


class Step:
    """The experts' part of a step, with every buffer its own."""

    def __init__(self, seed, rows=200, experts=4, hidden=96, inner=64, f8=True):
        self.x, self.dout = normal(seed, rows, hidden), normal(seed + 1, rows, hidden, sigma=0.01)
        self.up, self.down = normal(seed + 2, experts, hidden, 2 * inner, sigma=0.1), normal(seed + 3, experts, inner, hidden, sigma=0.1)
        self.bias = normal(seed + 4, experts, 2 * inner, dtype=torch.float32)
        self.offsets = offsets_of([0, 50, 50, 130, rows])
        self.f8 = fq.FQ_F8_MX if f8 else fq.FQ_F8_NONE

    def run(self, stream=None):
        rows, inner = self.x.shape[0], self.down.shape[1]
        new = lambda *s, dtype: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
        with torch.cuda.stream(stream) if stream else torch.cuda.stream(torch.cuda.current_stream()):
            pre = new(rows, 2 * inner, dtype=torch.uint8 if self.f8 else torch.bfloat16)
            scales = new(rows, 2 * inner // 32, dtype=torch.uint8) if self.f8 else None
            h2 = new(rows, inner, dtype=torch.bfloat16)
        kw = dict(offsets=self.offsets, stream=stream)
        kept = dict(pre_f8=self.f8, pre_scales=scales)
        h = fq.fq_glu_fwd(self.x, self.up, bias=self.bias, pre=pre, **kept, **kw)
        y = fq.fq_linear_fwd(h, self.down, res=self.x, **kw)
        codes, xs = fq.fq_f8_encode(self.x, fq.FQ_F8_MX, stream=stream)
        dh, _, _ = fq.fq_linear_bwd(self.dout, h, self.down, need_dw=False, need_dbias=False, **kw)
        dx, dup, dbias = fq.fq_glu_bwd(dh, codes, self.up, pre, x_f8=fq.FQ_F8_MX, x_scales=xs, h=h2, **kept, **kw)
        _, ddown, _ = fq.fq_linear_bwd(self.dout, h2, self.down, need_dx=False, need_dbias=False, dw_dtype=torch.float32, **kw)
        return h, y, dh, dx, dup, dbias, h2, ddown


def test_own_stream():
    """Calls on a stream of their own, which allocate for themselves, while the
    current stream makes and frees tensors of the same sizes."""
    step = Step(0)
    want = step.run()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        got = step.run(stream)
        for t in want:
            torch.full_like(t, 7)
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured():
    """Several replays, with eager calls of the same operators between them and
    new values in the same inputs."""
    step = Step(1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step.run()
    other = Step(9, rows=77, f8=False)
    other.offsets = offsets_of([0, 20, 30, 77, 77])
    for seed in (1, 5, 6, 7):
        fresh = Step(seed)
        step.x.copy_(fresh.x)
        step.dout.copy_(fresh.dout)
        step.up.copy_(fresh.up)
        step.down.copy_(fresh.down)
        step.bias.copy_(fresh.bias)
        starts = offsets_of([[0, 50, 50, 130, 200], [0, 0, 0, 0, 200], [0, 1, 2, 3, 200], [0, 199, 199, 200, 200]][seed % 4])
        step.offsets.copy_(starts)
        other.run()
        graph.replay()
        torch.cuda.synchronize()
        want = step.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed


def test_two_streams_at_once():
    """Two steps with their own workspaces, at the same time."""
    steps = [Step(2), Step(3, rows=201)]
    steps[1].offsets = offsets_of([0, 0, 201, 201, 201])
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = [s.run(st) for s, st in zip(steps, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,k,experts,f8", [(300, 2, 5, False), (300, 2, 5, True), (1, 4, 8, False), (64, 1, 3, False)])
def test_experts_of_a_step(tokens, k, experts, f8):
    """Norm, sort, dispatch, gated block, second projection, combine, and all of
    it backward, against autograd in 64 bits.

    Tolerance: each of the chain's BF16 roundings (y of the norm, rows, h, the
    second product, the combined rows; dy of the rows, dh, dz, dx of the rows, dx)
    adds an error of 2^-8 of a value at most, 2^-9 in the mean square, which the
    linear parts carry on unchanged: ten of them, below 10 * 2^-8 together.  A
    checkpoint of z in 8 bits adds 2^-4 of z at most, which reaches the gradients
    through the slope of the gate, at most 1.13, and in dw again through h: below
    2.3 * 2^-4."""
    hidden, inner = 64, 96
    x = normal(0, tokens, hidden)
    gamma = 1 + 0.1 * normal(1, hidden, dtype=torch.float32)
    up, down = normal(2, experts, hidden, 2 * inner, sigma=0.15), normal(3, experts, inner, hidden, sigma=0.15)
    bias = normal(4, experts, 2 * inner, sigma=0.2, dtype=torch.float32)
    ids = torch.stack([torch.randperm(experts, generator=torch.Generator().manual_seed(t))[:k] for t in range(tokens)]).int().to(DEV)
    weights = torch.softmax(normal(5, tokens, k, dtype=torch.float32), 1)
    dout = normal(6, tokens, hidden, sigma=0.01)

    rstd = torch.empty(tokens, device=DEV)
    _, y = fq.fq_rmsnorm_fwd(x, gamma, 1e-5, rstd=rstd)
    q = fq.fq_moe_sort(ids, experts, 1)
    rows = fq.fq_moe_dispatch(y, q)
    n = rows.shape[0]
    pre = torch.empty((n, 2 * inner), dtype=torch.uint8 if f8 else torch.bfloat16, device=DEV)
    kept = dict(pre_f8=fq.FQ_F8_MX, pre_scales=torch.empty((n, inner // 16), dtype=torch.uint8, device=DEV)) if f8 else {}
    h = fq.fq_glu_fwd(rows, up, bias=bias, offsets=q.offsets, pre=pre, **kept)
    out = fq.fq_linear_fwd(h, down, offsets=q.offsets)
    mixed = fq.fq_moe_combine(out, q, weights)
    drows, dweights = fq.fq_moe_combine_bwd(dout, out, q, weights)
    dh, _, _ = fq.fq_linear_bwd(drows, h, down, offsets=q.offsets, need_dw=False, need_dbias=False)
    again = torch.empty_like(h)
    dr, dup, dbias = fq.fq_glu_bwd(dh, rows, up, pre, offsets=q.offsets, h=again, **kept)
    _, ddown, _ = fq.fq_linear_bwd(drows, again, down, offsets=q.offsets, need_dx=False, need_dbias=False)
    dx, dgamma = fq.fq_rmsnorm_bwd(fq.fq_moe_combine(dr, q), x, gamma, rstd)
    torch.cuda.synchronize()

    leaves = [t.double().requires_grad_() for t in (x, gamma, up, bias, down, weights)]
    vx, vg, vu, vb, vd, vw = leaves
    yn = vx / torch.sqrt(vx.square().mean(1, keepdim=True) + 1e-5) * vg
    total = torch.zeros((tokens, hidden), dtype=torch.float64, device=DEV)
    for j in range(k):
        e = ids[:, j].long()
        z = torch.bmm(yn[:, None], vu[e])[:, 0] + vb[e]
        g, u = z.chunk(2, 1)
        total = total + vw[:, j:j + 1] * torch.bmm((torch.nn.functional.silu(g) * u)[:, None], vd[e])[:, 0]
    total.backward(dout.double())
    tol = 10 * 2.0 ** -8
    assert rel(mixed, total.detach()) < tol
    tol += 2.3 * 2.0 ** -4 if f8 else 0
    for name, got, leaf in (("dx", dx, vx), ("dgamma", dgamma, vg), ("dup", dup, vu), ("dbias", dbias, vb), ("ddown", ddown, vd),
                            ("dweights", dweights, vw)):
        assert rel(got, leaf.grad) < tol, (name, rel(got, leaf.grad))


def test_fake_quantized_operands():
    """The products of fake-quantized operands, as a quantized layer runs them:
    all experts' weights in one call, blocks along the contraction."""
    experts, k, n, rows = 3, 64, 96, 120
    x, w = normal(0, rows, k), normal(1, experts, k, 2 * n, sigma=0.1)
    xq = fq.fq_fake_quant(fq.fq_desc_mxfp4(), x)
    wq = fq.fq_fake_quant(fq.fq_desc_mxfp4(axis=fq.FQ_AXIS_COL), w.view(experts * k, 2 * n)).view(experts, k, 2 * n)
    starts = [0, 40, 41, 120]
    h = fq.fq_glu_fwd(xq, wq, offsets=offsets_of(starts))
    v, t = op.glu_fwd(xq, wq, None, (op.SILU, 1.0, math.inf, 0.0), starts)
    assert bool(((h.double() - v["y"]).abs() <= t["y"]).all())
    for e, (a, b) in enumerate(zip(starts, starts[1:])):
        same = fq.fq_qlinear_fwd(fq.fq_desc_mxfp4(), fq.fq_desc_mxfp4(axis=fq.FQ_AXIS_COL), x[a:b].contiguous(), w[e].contiguous())
        z, tz = op.linear_fwd(xq[a:b], wq[e], None, None, op.NONE)
        y = fq.fq_linear_fwd(xq[a:b].contiguous(), wq[e].contiguous())
        assert bool(((y.double() - z["y"]).abs() <= tz["y"]).all()) and bool(((same.double() - z["y"]).abs() <= tz["y"]).all())


# ---- the ends of the documented ranges ------------------------------------------------
# Small integers, so that every sum and rounding is exact.

def small_ints(seed, *shape, top):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_largest_values_before_silu(sign):
    """alpha z is infinite, z is not: a'(z) is 1 and 0, and a(z) is z and 0."""
    n = 32
    pre = torch.empty((4, 2 * n), dtype=torch.bfloat16, device=DEV)
    pre[:, :n] = sign * 3.3e38
    pre[:, n:] = 0.5
    dh = torch.ones((4, n), dtype=torch.bfloat16, device=DEV)
    h = torch.empty_like(dh)
    _, _, dbias = fq.fq_glu_bwd(dh, normal(0, 4, 32), normal(1, 32, 2 * n), pre, alpha=1.702, h=h, need_dx=False, need_dw=False)
    z = float(pre[0, 0])
    assert bool((dbias[:n] == (2.0 if sign > 0 else 0.0)).all())
    assert torch.equal(h.float(), torch.full_like(h, z / 2 if sign > 0 else 0.0).float().abs())


@pytest.mark.parametrize("rows,cols", [((1 << 24) + 3, 544), ((1 << 28) + 5, 32)])
def test_encode_more_rows_than_a_grid_axis(rows, cols):
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[:3], x[-3:] = normal(0, 3, cols), normal(1, 3, cols)
    codes, scales = fq.fq_f8_encode(x, fq.FQ_F8_ROW)
    for part in (slice(0, 4), slice(rows - 4, rows)):
        want, want_scales = op.encode_row(x[part])
        assert torch.equal(codes[part], want) and torch.equal(scales[part], want_scales)
    assert bool((scales[3:-3] == scales[3]).all())
    del x, codes, scales
    torch.cuda.empty_cache()


def test_few_rows_of_many_wide_experts():
    experts, k, n, each = 1024, 8, 1 << 18, 4
    x, w = small_ints(0, experts * each, k, top=3), small_ints(1, experts, k, n, top=3)
    starts = torch.arange(experts + 1, dtype=torch.int32, device=DEV) * each
    y = fq.fq_linear_fwd(x, w, offsets=starts)
    for e in range(0, experts, 64):
        want = torch.bmm(x.view(experts, each, k)[e: e + 64].float(), w[e: e + 64].float())
        assert torch.equal(y.view(experts, each, n)[e: e + 64].float(), want), e
    del x, w, y
    torch.cuda.empty_cache()


def test_gradients_of_many_wide_experts():
    """2^24 tiles: the widest weight of the most experts, two of which have rows."""
    experts, k, n, rows = 1024, 8, 1 << 20, 9
    x, dh = small_ints(0, rows, k, top=1), small_ints(1, rows, n, top=2)
    pre = torch.ones((rows, 2 * n), dtype=torch.bfloat16, device=DEV)
    pre[:, n:] = 2
    starts = torch.ones(experts + 1, dtype=torch.int32, device=DEV)
    starts[0], starts[-1] = 0, rows
    dw = torch.ones((experts, k, 2 * n), dtype=torch.bfloat16, device=DEV)
    fq.fq_glu_bwd(dh, x, dw, pre, act=fq.FQ_ACT_RELU, offsets=starts, dw=dw, need_dx=False, need_dbias=False)
    dz = torch.cat((2 * dh, dh), 1).float()
    assert torch.equal(dw[0].float(), x[:1].float().T @ dz[:1])
    assert torch.equal(dw[-1].float(), x[1:].float().T @ dz[1:])
    for e in range(1, experts - 1):
        assert not bool(dw[e].any()), e
    del dw
    torch.cuda.empty_cache()


def test_most_rows():
    rows = 1 << 30
    x = torch.zeros((rows, 8), dtype=torch.bfloat16, device=DEV)
    w = small_ints(0, 8, 8, top=3)
    at = [0, 1, 127, (1 << 29) + 3, rows - 129, rows - 1]
    for i, r in enumerate(at):
        x[r] = small_ints(i + 1, 8, top=3)
    y = fq.fq_linear_fwd(x, w)
    for r in at:
        assert torch.equal(y[r].float(), x[r].float() @ w.float()), r
    assert bool((y[2:127] == 0).all()) and bool((y[rows - 128: rows - 1] == 0).all())
    _, _, dbias = fq.fq_linear_bwd(x, y, w, need_dx=False, need_dw=False)
    assert torch.equal(dbias, x[at].float().sum(0))
    del x, y
    torch.cuda.empty_cache()
