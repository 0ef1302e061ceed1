"""AdamW with an eps at either end of FP32's range, where a hardware reciprocal
of sqrt(v) + eps leaves it: against float64."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("lr", [2.0 ** -20, 1.0])
@pytest.mark.parametrize("eps", [2.0 ** -149, 1e-40, 1e-38, 1e-30, 1e-8, 1.0, 1e30, 1e38, 3.4e38])
def test_any_eps(eps, lr, f8):
    """Elements that never had a gradient stay where they are, others take the
    formula's step: m * eps's reciprocal where v is 0.  The quotient's rounding
    and five more: 10 u."""
    n = 2051
    g = torch.logspace(-38, 5, n, device=DEV)
    g[::5] = 0
    t = fq.AdamWTensor(w=torch.zeros(n, device=DEV), g=g, **fq.adamw_state(n, DEV, f8))
    wide = fq.AdamWTensor(w=torch.zeros(n, device=DEV), g=g, **fq.adamw_state(n, DEV))
    hyper = dict(lr=lr, step=1, beta1=0.5, beta2=0.5, eps=eps)
    fq.fq_adamw_step(fq.adamw_plan([wide]), **hyper)
    fq.fq_adamw_step(fq.adamw_plan([t]), **hyper)
    assert (wide.w[::5] == 0).all()
    assert torch.equal(t.w, wide.w)
    m, v = wide.m.cpu().double().numpy(), wide.v.cpu().double().numpy()
    want = -2 * lr * m / (np.sqrt(v) * np.sqrt(2) + float(np.float32(eps)))
    got = wide.w.cpu().double().numpy()
    assert np.all(np.abs(got - want) <= 10 * U * np.abs(want) + 2.0 ** -148)
