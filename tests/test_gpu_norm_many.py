"""The norm of 512 rows and more, where half as many lanes have twice the chunks
(without a residual, and with one below 2^23 elements) and where calls stream
(from 2^24 elements on): every width class, against the formula in float64 on
the device.

Error bounds, u = 2^-24.  A lane adds at most 80 squares (10 chunks of 8), a row
22 further sums across lanes and waves; with the square's own rounding, the mean
and eps that is 105 u of the sum of squares, half of it in the root, and three
roundings more lead to r: within 64 u.  n is two products further, still within
64 u.  Backward: a lane adds at most 72 products (9 chunks), a row 22 sums, each
product has three roundings before it is added and the result six after: within
104 u of the sizes of its terms.  dgamma: (rows + 8) u of the sum of magnitudes.
BF16 adds half a step, 2^-8 of the value."""
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from test_gpu_norm import EPS, U, check_codes, f64
from test_gpu_norm_rows import guarded

pytestmark = pytest.mark.gpu

# 512 and 513 rows of each class: <64, 2> .. <512, 10>; the widest stream
FEW = [(512, 57), (513, 505), (512, 520), (513, 1000), (512, 1024), (513, 1056), (513, 1031), (512, 2048), (513, 2600),
       (512, 3001), (512, 4096), (513, 4090), (513, 6000), (512, 8185), (512, 8192), (513, 8188), (513, 16377), (512, 16384),
       (512, 16381), (513, 32761), (512, 32767), (513, 32768)]
# 2^24 elements and more
STREAMING = [(262147, 64), (131080, 129), (65600, 256), (33000, 512), (16400, 1024), (16411, 1031), (8200, 2048), (8211, 2047),
             (4100, 4096), (2763, 6072), (2100, 8185), (2051, 8192), (1027, 16383), (1030, 16384), (515, 32767)]


def values(rows, cols, stream, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device=DEV).to(torch.bfloat16)
    gamma = 1 + 0.2 * torch.randn(cols, generator=g, device=DEV)
    if stream == "none":
        return g, x, None, gamma, x
    res = torch.randn((rows, cols), generator=g, device=DEV) * 2
    res[:, :2] *= 50
    res = res if stream == "f32" else res.to(torch.bfloat16)
    # the sum in FP32, then the stream's type
    return g, x, res, gamma, (x.float() + res.float()).to(res.dtype)


def norm64(h, gamma):
    h = h.double()
    r = (h.square().mean(1) + float(torch.tensor(EPS, dtype=torch.float32))).rsqrt()
    return h * r[:, None] * gamma.double(), r


@pytest.mark.parametrize("rows, cols", FEW + STREAMING)
@pytest.mark.parametrize("stream", ["none", "bf16", "f32"])
def test_forward(rows, cols, stream):
    _, x, res, gamma, h = values(rows, cols, stream, rows + cols)
    y, around_y = guarded(rows, cols, torch.bfloat16)
    hg, around_h = guarded(rows, cols, h.dtype)
    rstd = torch.empty(rows, device=DEV)
    fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, h=None if res is None else hg, y=y, rstd=rstd)
    n, r = norm64(h, gamma)
    if res is not None:
        assert torch.equal(hg, h)
    assert ((rstd.double() - r).abs() <= 64 * U * r).all()
    assert ((y.double() - n).abs() <= (2.0 ** -8 + 64 * U) * n.abs()).all()
    assert all((t == 7).all() for t in around_y + (around_h if res is not None else ()))


@pytest.mark.parametrize("rows, cols", [(513, 32), (512, 544), (513, 1024), (512, 1056), (513, 2048), (513, 2592), (512, 4096),
                                        (513, 6016), (512, 8192), (512, 16384), (513, 32768), (16400, 1024), (2051, 8192)])
@pytest.mark.parametrize("f8", [fq.FQ_F8_MX, fq.FQ_F8_ROW])
@pytest.mark.parametrize("stream", ["none", "bf16", "f32"])
def test_forward_8bit(rows, cols, f8, stream):
    _, x, res, gamma, h = values(rows, cols, stream, cols)
    y, around_y = guarded(rows, cols, torch.bfloat16)
    codes, around_c = guarded(rows, cols, torch.uint8)
    _, _, scales = fq.fq_rmsnorm_fwd(x, gamma, EPS, res=res, f8=f8, y=y, codes=codes)
    v = check_codes(f64(norm64(h, gamma)[0]), codes, scales, f8, cols)
    v = torch.tensor(v, device=DEV)
    # a power of two's values are BF16 numbers; an FP32 scale's are rounded
    half = 0.0 if f8 == fq.FQ_F8_MX else 2.0 ** -8 + U
    assert ((y.double() - v).abs() <= half * v.abs()).all()
    assert all((t == 7).all() for t in around_y + around_c)


@pytest.mark.parametrize("rows, cols", STREAMING + [(513, 32768)])
@pytest.mark.parametrize("stream", ["none", "bf16", "f32"])
def test_backward(rows, cols, stream):
    g, _, _, gamma, h = values(rows, cols, stream, rows)
    rstd = norm64(h, gamma)[1].float()
    dy = (torch.randn((rows, cols), generator=g, device=DEV) * 1e-3).to(torch.bfloat16)
    dres = None if stream == "none" else (torch.randn((rows, cols), generator=g, device=DEV) * 1e-3).to(h.dtype)
    dh, around = guarded(rows, cols, h.dtype)
    dx, around_x = guarded(rows, cols, torch.bfloat16)
    _, dgamma = fq.fq_rmsnorm_bwd(dy, h, gamma, rstd, dres=dres, dh=dh, dx=dx)
    r = rstd.double()[:, None]
    xh, gg = h.double() * r, dy.double() * gamma.double()
    size = r * (gg.abs() + xh.abs() * (gg * xh).abs().mean(1, keepdim=True))
    want = r * (gg - xh * (gg * xh).mean(1, keepdim=True))
    want = want if dres is None else want + dres.double()
    half = U if h.dtype == torch.float32 else 2.0 ** -8
    fp32 = 104 * U * size + 2 * U * want.abs()
    assert ((dh.double() - want).abs() <= half * want.abs() + (1 + half) * fp32).all()
    # the BF16 copy is rounded from FP32 once
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1.01 * fp32).all()
    p = dy.double() * xh
    assert ((dgamma.double() - p.sum(0)).abs() <= (rows + 8) * U * p.abs().sum(0)).all()
    assert all((t == 7).all() for t in around + around_x)
