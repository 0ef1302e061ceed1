"""Every shape of tiles that the feed-forward products choose from, dense and over
experts' segments, with values checked against the oracle: residuals and biases of
several experts, values kept in BF16 and 8 bits, and contractions of segments from
none to many stages.

The sizes are the smallest of their kind for which the launchers' rules take the
shapes named beside them (128x128 in two or four stages as /2 and /4)."""
import pytest
import torch

from oracle import products as op
from test_gpu_products import run_bwd, run_glu, run_linear

pytestmark = pytest.mark.gpu

# Lengths around a tile's rows, a stage's 64 k, and the ends of two, three and four
# stages' pipelines; the last segment takes what is left but `tail` rows.
LENGTHS = [63, 0, 1, 257, 129, 64, 340, 192]


def uneven(rows, experts, tail=7):
    starts = [0]
    for e in range(experts - 1):
        room = rows - tail - starts[-1]
        starts.append(starts[-1] + min(LENGTHS[e % len(LENGTHS)], room))
    return starts + [rows - tail]


# rows, k, n, experts (0: dense)
LINEAR = [(1030, 392, 264, 6),            # 128x128/4
          (1030, 392, 2056, 8),           # 128x128/2
          (1500, 392, 4104, 8),           # 256x192
          (2100, 392, 4104, 8),           # 256x256
          (1500, 392, 4104, 0),           # 128x128/2
          (2050, 392, 4128, 0),           # 256x192
          (4090, 392, 4088, 0)]           # 256x256


@pytest.mark.parametrize("rows,k,n,experts", LINEAR)
@pytest.mark.parametrize("out,inplace,bias", [(torch.bfloat16, False, torch.float32), (torch.float32, False, torch.bfloat16),
                                              (torch.bfloat16, True, torch.bfloat16), (torch.float32, True, None)])
def test_bias_and_residual(rows, k, n, experts, out, inplace, bias):
    run_linear(rows, k, n, uneven(rows, experts) if experts else None, out=out, inplace=inplace, bias=bias)


@pytest.mark.parametrize("rows,k,n,experts", [
    (1030, 392, 288, 6),                  # 128x128/4
    (1030, 392, 2080, 8),                 # 128x128/2
    (1500, 392, 4128, 8),                 # 256x192
    (2100, 392, 4128, 8),                 # 256x256
    (2050, 392, 4128, 0),                 # 256x192
    (4090, 392, 4064, 0)])                # 256x256
@pytest.mark.parametrize("act,pre,out", [(op.GELU, "mx", torch.bfloat16), (op.SILU, "bf16", torch.float32), (op.NONE, "mx", torch.float32),
                                         (op.RELU, "none", torch.bfloat16)])
def test_activation_and_kept_values(rows, k, n, experts, act, pre, out):
    run_linear(rows, k, n, uneven(rows, experts) if experts else None, act=act, pre=pre, out=out, res=act != op.GELU)


@pytest.mark.parametrize("rows,k,n,experts", [
    (1030, 392, 288, 4),                  # 128x64/4
    (2100, 392, 1056, 8),                 # 128x64/2
    (5000, 392, 800, 5),                  # 256x128
    (5000, 392, 800, 0),                  # 256x128
    (2100, 392, 2080, 0)])                # 256x128
@pytest.mark.parametrize("gate,pre", [("clamped", "mx"), ("gelu", "bf16"), ("silu", "none")])
def test_gated(rows, k, n, experts, gate, pre):
    run_glu(rows, k, n, uneven(rows, experts) if experts else None, gate=gate, pre=pre)


@pytest.mark.parametrize("rows,k,n,experts,gate", [
    (1150, 264, 520, 6, "clamped"),       # dx 128x128, dw 128x128
    (1150, 136, 2056, 8, "silu"),         # dx 128x128, dw 192x192
    (1150, 3080, 136, 8, "clamped"),      # dx 128x128, dw 256x256
    (2100, 4104, 136, 8, None),           # dx 256x256, dw 192x192
    (2100, 4104, 200, 9, None),           # dx 256x256, dw 256x256
    (2100, 3080, 264, 9, None),           # dx 256x192, dw 256x256
    (2700, 2872, 136, 8, "silu"),         # dx 256x192, dw 192x192
    (3000, 4104, 456, 0, None),           # dx 256x256, dw 128x128
    (2100, 4104, 1032, 0, "clamped")])    # dx 256x192, dw 192x192
@pytest.mark.parametrize("dw_dtype", [torch.bfloat16, torch.float32])
def test_backward(rows, k, n, experts, gate, dw_dtype):
    run_bwd(rows, k, n, uneven(rows, experts) if experts else None, gate=gate, act=op.GELU, dw_dtype=dw_dtype)


@pytest.mark.parametrize("rows,k,n,experts", [
    (3000, 2880, 160, 8),                 # dx 256x192, dw 192x192
    (3000, 3104, 160, 8)])                # dx 256x256, dw 256x256
@pytest.mark.parametrize("x_how", ["mx", "row"])
def test_backward_from_8_bits(rows, k, n, experts, x_how):
    run_bwd(rows, k, n, uneven(rows, experts), gate="clamped", x_how=x_how, pre_how="mx", dw_dtype=torch.float32)
