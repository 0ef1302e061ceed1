"""The feed-forward products against the oracle in 64 bits, element by element
within bounds that follow from the formulas (oracle/products.py)."""
import math

import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from oracle import products as op
from product_util import Guarded, normal, offsets_of, pre_buffers, untouched, within

pytestmark = pytest.mark.gpu

GATES = {"silu": (op.SILU, 1.0, math.inf, 0.0), "gelu": (op.GELU, 1.0, math.inf, 0.0),
         "clamped": (op.SILU, 1.702, 1.25, 1.0), "relu": (op.RELU, 1.0, math.inf, 0.0),
         "none": (op.NONE, 1.0, 2.0, 0.5)}


def gate_args(name):
    return dict(zip(("act", "alpha", "limit", "shift"), GATES[name]))


def spread(rows, experts, seed=0, tail=0):
    """Segments of very different lengths, some empty, `tail` rows behind them."""
    g = torch.Generator().manual_seed(seed)
    like = torch.rand(experts, generator=g) ** 3 * (torch.rand(experts, generator=g) > 0.25)
    if float(like.sum()) == 0:
        like[-1] = 1
    ends = (torch.cumsum(like, 0) / like.sum() * (rows - tail)).round().long()
    ends[-1] = rows - tail
    return [0] + ends.tolist()


def check_pre(pre, scales, z, tz, kind):
    if kind == "bf16":
        within(pre, z, tz + op.EPS16 * (z.abs() + tz) + op.FLOOR, "pre")
    elif kind == "mx":
        b = z.reshape(z.shape[0], -1, 32)
        t = tz.reshape(b.shape)
        low, high = (op.encode_mx((b.abs().amax(2, keepdim=True) + s * t.amax(2, keepdim=True)).expand(b.shape).reshape(z.shape))[1]
                     for s in (-1, 1))
        assert bool(((scales >= low) & (scales <= high)).all()), "scales"
        s = op.pow2(scales.long() - 127).repeat_interleave(32, 1)
        within(op.decode(pre, scales, True), z, tz + 2.0 ** -4 * (z.abs() + tz) + 2.0 ** -10 * s, "pre in 8 bits")


def run_linear(rows, k, n, starts=None, act=op.NONE, out=torch.bfloat16, res=True, pre="none", bias=torch.float32, inplace=False, seed=0):
    lead = () if starts is None else (len(starts) - 1,)
    g = Guarded()
    x = g.input(normal(seed, rows, k))
    end = rows if starts is None else starts[-1]
    x[end:] = math.nan
    w = g.input(normal(seed + 1, *lead, k, n, sigma=k ** -0.5))
    b = None if bias is None else g.input(normal(seed + 2, *lead, n, dtype=bias))
    r = normal(seed + 3, rows, n, dtype=out) if res else None
    y = g.output((rows, n), out)
    if inplace:
        y[:end] = r[:end]
    p, f8, scales = pre_buffers(g, rows, n, pre)
    fq.fq_linear_fwd(x, w, bias=b, res=y if inplace else g.input(r), act=act, offsets=offsets_of(starts), pre=p, pre_f8=f8,
                     pre_scales=scales, y=y)
    torch.cuda.synchronize()
    g.check()
    v, t = op.linear_fwd(x, w, b, r, act, starts, out)
    within(y[:end], v["y"][:end], t["y"][:end], "y")
    if p is not None:
        check_pre(p[:end], None if scales is None else scales[:end], v["z"][:end], t["z"][:end], pre)
        assert untouched(p[end:]) and (scales is None or untouched(scales[end:]))
    assert untouched(y[end:]), "rows behind the last segment"


# one token, ragged rows, odd multiples of eight, contractions that end inside a step; the last ones take the large tiles
SHAPES = [(1, 8, 8), (1, 72, 264), (1, 2880, 200), (2, 64, 64), (3, 1000, 136), (7, 520, 1032), (16, 128, 72), (17, 136, 128), (31, 64, 8),
          (33, 200, 320), (64, 1032, 96), (65, 264, 392), (127, 8, 128), (128, 192, 256), (129, 64, 264), (257, 776, 136),
          (300, 40, 1096), (1021, 72, 776), (4200, 72, 4168), (4090, 72, 4088), (4090, 392, 4088), (4200, 456, 4168), (4090, 392, 2040),
          # wide weights of few rows, contractions in parts, four stages
          (1, 72, 8200), (17, 72, 8200), (40, 264, 8200), (64, 136, 8200), (100, 1032, 136), (200, 2880, 264), (130, 4104, 72),
          (1900, 1032, 1896)]


@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_linear(rows, k, n):
    run_linear(rows, k, n)


@pytest.mark.parametrize("act", [op.NONE, op.RELU, op.SILU, op.GELU])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,pre", [(1, "bf16"), (5, "mx"), (77, "mx"), (77, "none"), (150, "bf16")])
def test_linear_epilogues(act, out, rows, pre):
    run_linear(rows, 72, 160, act=act, out=out, pre=pre, res=act != op.GELU, bias=torch.bfloat16 if rows == 5 else torch.float32)


def test_linear_bare():
    run_linear(150, 64, 136, res=False, bias=None)
    run_linear(3, 64, 136, res=False, bias=None)


@pytest.mark.parametrize("act", [op.NONE, op.SILU])
@pytest.mark.parametrize("pre", ["bf16", "mx"])
def test_epilogues_of_joined_parts(act, pre):
    run_linear(100, 1032, 160, act=act, pre=pre)
    run_linear(100, 1032, 160, act=act, out=torch.float32, pre=pre, bias=torch.bfloat16)
    run_linear(100, 1032, 160, act=act, inplace=True)
    run_glu(100, 1032, 160, gate="clamped" if act else "gelu", pre=pre)


@pytest.mark.parametrize("rows", [1, 17, 40])
def test_few_rows_of_wide_weights(rows):
    run_linear(rows, 72, 8224, act=op.GELU, pre="mx", out=torch.float32)
    run_glu(rows, 72, 8224, gate="clamped", pre="mx")


@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_linear_in_place(rows, out):
    run_linear(rows, 136, 264, out=out, inplace=True, act=op.SILU)


@pytest.mark.parametrize("rows,k,n,experts,tail", [
    (1, 64, 64, 1, 0), (1, 72, 136, 5, 0), (9, 72, 136, 4, 2), (40, 200, 72, 7, 0), (130, 264, 136, 3, 13), (600, 72, 264, 32, 0),
    (600, 136, 200, 130, 5), (1500, 64, 1032, 4, 100), (5000, 72, 1544, 5, 8)])
def test_linear_experts(rows, k, n, experts, tail):
    run_linear(rows, k, n, spread(rows, experts, rows, tail), act=op.SILU)


@pytest.mark.parametrize("starts", [[0, 0, 0, 0], [0, 0, 300, 300], [0, 300, 300, 300], [0, 1, 2, 3], [0, 127, 128, 300], [0, 16, 32, 33]])
def test_linear_segments(starts):
    run_linear(300, 72, 136, starts, pre="bf16")


def run_glu(rows, k, n, starts=None, gate="silu", pre="none", bias=torch.float32, seed=0):
    lead = () if starts is None else (len(starts) - 1,)
    g = Guarded()
    end = rows if starts is None else starts[-1]
    x = g.input(normal(seed, rows, k))
    x[end:] = math.nan
    w = g.input(normal(seed + 1, *lead, k, 2 * n, sigma=k ** -0.5))
    b = None if bias is None else g.input(normal(seed + 2, *lead, 2 * n, dtype=bias))
    h = g.output((rows, n), torch.bfloat16)
    p, f8, scales = pre_buffers(g, rows, 2 * n, pre)
    fq.fq_glu_fwd(x, w, bias=b, offsets=offsets_of(starts), pre=p, pre_f8=f8, pre_scales=scales, h=h, **gate_args(gate))
    torch.cuda.synchronize()
    g.check()
    v, t = op.glu_fwd(x, w, b, GATES[gate], starts)
    within(h[:end], v["y"][:end], t["y"][:end], "h")
    if p is not None:
        check_pre(p[:end], None if scales is None else scales[:end], v["z"][:end], t["z"][:end], pre)
        assert untouched(p[end:]) and (scales is None or untouched(scales[end:]))
    assert untouched(h[end:]), "rows behind the last segment"


@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_glu(rows, k, n):
    run_glu(rows, k, n)


@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("rows,pre", [(1, "mx"), (6, "bf16"), (70, "mx"), (140, "bf16"), (140, "none")])
def test_glu_epilogues(gate, rows, pre):
    run_glu(rows, 72, 160, gate=gate, pre=pre, bias=torch.bfloat16 if rows == 6 else torch.float32 if rows > 1 else None)


@pytest.mark.parametrize("rows,k,n,experts,tail", [
    (1, 64, 64, 1, 0), (1, 72, 136, 5, 0), (9, 72, 96, 4, 2), (130, 264, 136, 3, 13), (600, 72, 264, 32, 0),
    (600, 136, 200, 130, 5), (1500, 64, 776, 4, 100), (5000, 72, 1032, 5, 8)])
def test_glu_experts(rows, k, n, experts, tail):
    run_glu(rows, k, n, spread(rows, experts, rows, tail), gate="clamped", pre="bf16" if n % 32 else "mx")


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------

def kept(g, v, how):
    """(tensor for the call, f8, scales, the BF16 values it stands for)."""
    if how == "bf16":
        return g.input(v), fq.FQ_F8_NONE, None, v
    codes, scales = op.encode_mx(v) if how == "mx" else op.encode_row(v)
    value = op.decode(codes, scales, how == "mx")
    # FP32 product of code and scale, rounded to BF16
    return g.input(codes), fq.FQ_F8_MX if how == "mx" else fq.FQ_F8_ROW, g.input(scales), value.float().to(torch.bfloat16)


def run_bwd(rows, k, n, starts=None, gate=None, act=op.NONE, x_how="bf16", pre_how="bf16", dw_dtype=torch.bfloat16, with_h=True, seed=0):
    halves = 2 if gate else 1
    cols = n * halves
    lead = () if starts is None else (len(starts) - 1,)
    end = rows if starts is None else starts[-1]
    g = Guarded()
    dy = g.input(normal(seed, rows, n, sigma=0.01))
    x, x_f8, x_scales, xv = kept(g, normal(seed + 1, rows, k), x_how)
    if x_how == "row" and (gate or act != op.NONE):
        # not rounded by itself, but together with dz, whose bound has that rounding
        xv = op.decode(x, x_scales, False)
    w = g.input(normal(seed + 2, *lead, k, cols, sigma=k ** -0.5))
    p, p_f8, p_scales, pv = (None, fq.FQ_F8_NONE, None, None) if not gate and act == op.NONE else kept(g, normal(seed + 3, rows, cols, sigma=1.5), pre_how)
    dy[end:] = math.nan
    if x_how == "bf16":
        x[end:] = math.nan
    if p is not None and pre_how == "bf16":
        p[end:] = math.nan
    dx, dw = g.output((rows, k), torch.bfloat16), g.output((*lead, k, cols), dw_dtype)
    db = g.output((*lead, cols), torch.float32)
    common = dict(offsets=offsets_of(starts), x_f8=x_f8, x_scales=x_scales, pre_f8=p_f8, pre_scales=p_scales, dx=dx, dw=dw, dbias=db)
    if gate:
        h = g.output((rows, n), torch.bfloat16) if with_h else None
        fq.fq_glu_bwd(dy, x, w, p, h=h, **gate_args(gate), **common)
        v, t = op.glu_bwd(dy[:end], xv[:end], w, pv[:end], GATES[gate], starts, dw_dtype)
    else:
        h = None
        fq.fq_linear_bwd(dy, x, w, pre=p, act=act, **common)
        v, t = op.linear_bwd(dy[:end], xv[:end], w, None if pv is None else pv[:end], act, starts, dw_dtype)
    torch.cuda.synchronize()
    g.check()
    within(dx[:end], v["dx"], t["dx"], "dx")
    within(dw, v["dw"], t["dw"], "dw")
    within(db, v["dbias"], t["dbias"], "dbias")
    assert untouched(dx[end:])
    if h is not None:
        within(h[:end], v["h"], t["h"], "h")
        assert untouched(h[end:])


BWD_SHAPES = [(1, 8, 8), (1, 264, 136), (2, 64, 64), (5, 1000, 72), (63, 72, 264), (64, 128, 128), (65, 136, 264), (100, 520, 776),
              (129, 256, 136), (333, 1000, 72), (1000, 72, 136), (2200, 4168, 136),
              (4090, 4088, 72), (4200, 4168, 72), (4200, 4168, 456), (100, 4088, 4088), (100, 2872, 2864), (456, 2872, 2864), (392, 4088, 4088),
              (100, 136, 2088), (2056, 136, 200), (1100, 200, 1160), (1900, 1896, 1032)]


@pytest.mark.parametrize("rows,k,n", BWD_SHAPES)
@pytest.mark.parametrize("dw_dtype", [torch.bfloat16, torch.float32])
def test_linear_bwd(rows, k, n, dw_dtype):
    run_bwd(rows, k, n, dw_dtype=dw_dtype)


@pytest.mark.parametrize("rows,k,n", [(1, 32, 8), (37, 96, 136), (300, 288, 72)])
def test_row_scales_without_activation(rows, k, n):
    run_bwd(rows, k, n, x_how="row")
    run_bwd(rows, k, n, spread(rows, 3, rows, rows // 9), x_how="row", dw_dtype=torch.float32)


@pytest.mark.parametrize("rows,k,n", [(1, 32, 8), (37, 96, 136), (300, 288, 72), (900, 2048, 520)])
@pytest.mark.parametrize("gate", [None, "clamped"])
def test_row_scales_are_rounded_with_dz(rows, k, n, gate):
    """FP32 dw from x with a scale per row: beside the bound of every element, its root
    mean square error is that of one rounding to BF16.  That is off by a uniform share of
    half a step, which is 2^-9 to 2^-8 of the value: 2^-8 / sqrt 3 = 0.00226 in the mean
    at most, 0.0017 for values of every mantissa; two roundings would have 0.0024."""
    run_bwd(rows, k, n, gate=gate, act=op.SILU, x_how="row")
    run_bwd(rows, k, n, spread(rows, 3, rows, rows // 9), gate=gate, act=op.SILU, x_how="row", dw_dtype=torch.float32)
    dy, x, w, pre = normal(0, rows, n), normal(1, rows, k), normal(2, k, n * (2 if gate else 1)), normal(3, rows, n * (2 if gate else 1))
    codes, scales = fq.fq_f8_encode(x, fq.FQ_F8_ROW)
    common = dict(x_f8=fq.FQ_F8_ROW, x_scales=scales, dw_dtype=torch.float32, need_dx=False, need_dbias=False)
    xv = op.decode(codes, scales, False)
    if gate:
        _, dw, _ = fq.fq_glu_bwd(dy, codes, w, pre, **gate_args(gate), **common)
        want = op.glu_bwd(dy, xv, w, pre, GATES[gate])[0]["dw"]
    else:
        _, dw, _ = fq.fq_linear_bwd(dy, codes, w, pre=pre, act=op.SILU, **common)
        want = op.linear_bwd(dy, xv, w, pre, op.SILU)[0]["dw"]
    if rows * n > 1000:
        assert float((dw.double() - want).norm() / want.norm()) <= 2.0 ** -8 / 3 ** 0.5 * 1.01


@pytest.mark.parametrize("act", [op.RELU, op.SILU, op.GELU])
@pytest.mark.parametrize("x_how", ["bf16", "mx", "row"])
@pytest.mark.parametrize("pre_how", ["bf16", "mx"])
def test_linear_bwd_kept(act, x_how, pre_how):
    run_bwd(150, 96, 160, act=act, x_how=x_how, pre_how=pre_how, dw_dtype=torch.float32)


@pytest.mark.parametrize("rows,k,n", BWD_SHAPES)
def test_glu_bwd(rows, k, n):
    run_bwd(rows, k, n, gate="silu")


@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("x_how,pre_how", [("bf16", "bf16"), ("mx", "mx"), ("row", "mx")])
def test_glu_bwd_kept(gate, x_how, pre_how):
    run_bwd(150, 96, 160, gate=gate, x_how=x_how, pre_how=pre_how, dw_dtype=torch.float32, with_h=x_how != "row")


@pytest.mark.parametrize("rows,k,n,experts,tail", [
    (1, 64, 64, 1, 0), (1, 72, 136, 5, 0), (9, 72, 136, 4, 2), (130, 264, 136, 3, 13), (600, 72, 264, 32, 0),
    (600, 136, 200, 130, 5), (1500, 264, 776, 4, 100), (5000, 72, 520, 5, 8)])
@pytest.mark.parametrize("gate", [None, "clamped"])
def test_experts_bwd(rows, k, n, experts, tail, gate):
    run_bwd(rows, k, n, spread(rows, experts, rows, tail), gate=gate, act=op.SILU)


@pytest.mark.parametrize("starts", [[0, 0, 0, 0], [0, 0, 300, 300], [0, 300, 300, 300], [0, 1, 2, 3], [0, 63, 65, 300], [0, 64, 128, 129]])
def test_segments_bwd(starts):
    run_bwd(300, 72, 136, starts, gate="silu")
    run_bwd(300, 72, 136, starts, x_how="bf16", dw_dtype=torch.float32)


def test_parts_of_the_backward():
    """Each output alone is what all of them together are."""
    dy, x, w = normal(0, 100, 136, sigma=0.01), normal(1, 100, 72), normal(2, 72, 272, sigma=0.1)
    pre = normal(3, 100, 272)
    all_of = fq.fq_glu_bwd(dy, x, w, pre)
    for i, name in enumerate(("need_dx", "need_dw", "need_dbias")):
        need = {n: n == name for n in ("need_dx", "need_dw", "need_dbias")}
        part = fq.fq_glu_bwd(dy, x, w, pre, **need)
        assert torch.equal(part[i], all_of[i]) and all(p is None for j, p in enumerate(part) if j != i)
    h = torch.empty((100, 136), dtype=torch.bfloat16, device=DEV)
    fq.fq_glu_bwd(dy, x, w, pre, h=h, need_dx=False, need_dw=False, need_dbias=False)
    v, t = op.glu_bwd(dy, x, w, pre, GATES["silu"])
    within(h, v["h"], t["h"], "h")


# ---------------------------------------------------------------------------
# values that are not finite, and what they may reach
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,k,n", [(5, 72, 136), (150, 72, 136), (150, 136, 264)])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_not_finite(rows, k, n, bad):
    """An infinity or NaN of x stays in its row, of w in its column; the zeros
    behind the end of the contraction meet none of them."""
    x, w = normal(0, rows, k), normal(1, k, n)
    x[rows - 1, k - 1] = bad
    w[k - 1, 3] = bad
    y = fq.fq_linear_fwd(x, w)
    torch.cuda.synchronize()
    fine = torch.isfinite(y)
    assert bool(fine[: rows - 1, :3].all()) and bool(fine[: rows - 1, 4:].all())
    assert not bool(fine[rows - 1].any()) and not bool(fine[:, 3].any())
    want = torch.where(w[k - 1].double() * bad > 0, math.inf, -math.inf)
    if math.isinf(bad):
        keep = torch.arange(n, device=DEV) != 3
        assert torch.equal(y[rows - 1].double()[keep], want[keep])
    dy = normal(2, rows, n)
    dy[rows - 1, n - 1] = bad
    dx, dw, db = fq.fq_linear_bwd(dy, normal(0, rows, k), normal(1, k, n), dw_dtype=torch.float32)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(dx[: rows - 1]).all()) and not bool(torch.isfinite(dx[rows - 1]).any())
    assert bool(torch.isfinite(dw[:, : n - 1]).all()) and not bool(torch.isfinite(dw[:, n - 1]).any())
    assert bool(torch.isfinite(db[: n - 1]).all()) and not bool(torch.isfinite(db[n - 1]))


def test_neighbours_of_a_segment_do_not_reach_it():
    """A NaN in one expert's last row leaves the next expert's results alone."""
    starts = [0, 70, 141, 300]
    x, w, dy = normal(0, 300, 72), normal(1, 3, 72, 136), normal(2, 300, 136)
    x[69] = math.nan
    dy[141] = math.nan
    y = fq.fq_linear_fwd(x, w, offsets=offsets_of(starts))
    dx, dw, db = fq.fq_linear_bwd(dy, x, w, offsets=offsets_of(starts))
    torch.cuda.synchronize()
    bad = torch.zeros(300, dtype=torch.bool, device=DEV)
    bad[69] = True
    assert torch.equal(torch.isnan(y).any(1), bad)
    assert torch.equal(torch.isnan(dw).flatten(1).any(1).cpu(), torch.tensor([True, False, True]))
    assert torch.equal(torch.isnan(db).any(1).cpu(), torch.tensor([False, False, True]))


def test_offsets_that_do_not_ascend_stay_inside():
    """Entries are brought into 0 .. rows: nothing is read or written outside."""
    for starts in ([-5, 40, 1 << 30], [90, 10, 100], [-(1 << 31), (1 << 31) - 1, 0], [100, 100, 100]):
        g = Guarded()
        x, w, dy = g.input(normal(0, 100, 72)), g.input(normal(1, 2, 72, 136)), g.input(normal(2, 100, 136))
        y, dx = g.output((100, 136), torch.bfloat16), g.output((100, 72), torch.bfloat16)
        dw, db = g.output((2, 72, 136), torch.float32), g.output((2, 136), torch.float32)
        fq.fq_linear_fwd(x, w, offsets=offsets_of(starts), y=y)
        fq.fq_linear_bwd(dy, x, w, offsets=offsets_of(starts), dx=dx, dw=dw, dbias=db)
        torch.cuda.synchronize()
        g.check()


@pytest.mark.parametrize("rows,experts", [(100, 600), (1000, 1024), (65, 1)])
def test_many_segments_that_overlap_stay_inside(rows, experts):
    """More tiles in the offsets than any that ascend have: no index leaves the
    outputs or the workspace, which ends where it has to."""
    starts = [0 if e % 2 == 0 else rows for e in range(experts + 1)]
    g = Guarded()
    x, w, dy = g.input(normal(0, rows, 64)), g.input(normal(1, experts, 64, 128)), g.input(normal(2, rows, 64))
    pre = g.input(normal(3, rows, 128))
    h, dx = g.output((rows, 64), torch.bfloat16), g.output((rows, 64), torch.bfloat16)
    dw, db = g.output((experts, 64, 128), torch.bfloat16), g.output((experts, 128), torch.float32)
    size = fq.glu_bwd_workspace(rows, 64, 64, experts, "cpu").numel()
    fq.fq_glu_fwd(x, w, offsets=offsets_of(starts), h=h)
    fq.fq_glu_bwd(dy, x, w, pre, offsets=offsets_of(starts), dx=dx, dw=dw, dbias=db, ws=g.output((size,), torch.uint8))
    torch.cuda.synchronize()
    g.check()


def test_equal_calls_give_equal_bits():
    starts = offsets_of(spread(700, 9, 3))
    x, w, dy, pre = normal(0, 700, 264), normal(1, 9, 264, 272), normal(2, 700, 136), normal(3, 700, 272)
    first = fq.fq_glu_bwd(dy, x, w, pre, offsets=starts)
    y = fq.fq_glu_fwd(x, w, offsets=starts)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, fq.fq_glu_bwd(dy, x, w, pre, offsets=starts)))
        assert torch.equal(y[: int(starts[-1])], fq.fq_glu_fwd(x, w, offsets=starts)[: int(starts[-1])])
