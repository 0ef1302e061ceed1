"""What the tests of the feed-forward products share: operands in guarded
memory, and the comparison with the oracle's results and bounds."""
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV

GUARD = 512                       # elements before and behind an operand


def normal(seed, *shape, sigma=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(dtype)


class Guarded:
    """Tensors inside larger buffers: inputs between NaN (0xFF bytes), outputs
    between bytes that have to stay."""

    def __init__(self):
        self.held = []

    def input(self, t):
        if t is None:
            return None
        raw = torch.full(((t.numel() + 2 * GUARD) * t.element_size(),), 0xFF, dtype=torch.uint8, device=DEV)
        v = raw[GUARD * t.element_size(): (GUARD + t.numel()) * t.element_size()].view(t.dtype).view(t.shape)
        v.copy_(t)
        return v

    def output(self, shape, dtype, fill=0x5A):
        n = torch.Size(shape).numel()
        size = torch.empty((), dtype=dtype).element_size()
        raw = torch.full(((n + 2 * GUARD) * size,), fill, dtype=torch.uint8, device=DEV)
        self.held.append((raw, GUARD * size, (GUARD + n) * size, fill))
        return raw[GUARD * size: (GUARD + n) * size].view(dtype).view(shape)

    def check(self):
        for raw, a, b, fill in self.held:
            assert bool((raw[:a] == fill).all()) and bool((raw[b:] == fill).all()), "written outside an output"


def untouched(t, fill=0x5A):
    return bool((t.contiguous().view(torch.uint8) == fill).all())


def within(got, want, bound, name):
    """Every element within its bound (and NaN nowhere)."""
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (
        f"{name}: {int(bad.sum())} of {bad.numel()} outside; first at {bad.nonzero()[0].tolist()}: "
        f"got {float(got[tuple(bad.nonzero()[0])])}, want {float(want[tuple(bad.nonzero()[0])])} "
        f"to {float(bound[tuple(bad.nonzero()[0])])}")


def offsets_of(starts):
    return None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)


def pre_buffers(g, rows, cols, kind):
    """(pre, pre_f8, pre_scales) of a forward."""
    if kind == "none":
        return None, fq.FQ_F8_NONE, None
    if kind == "bf16":
        return g.output((rows, cols), torch.bfloat16), fq.FQ_F8_NONE, None
    return g.output((rows, cols), torch.uint8), fq.FQ_F8_MX, g.output((rows, cols // 32), torch.uint8)
