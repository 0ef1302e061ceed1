"""An AdamW plan that is dropped right after a step on another stream than its
own: its table stays what it is until that step has run."""
import pytest
import torch

import fp4_block_quantization_fq_amd as fq
from gpu_util import DEV
from test_gpu_adamw import HYPER, check_f32, copy_of, tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("named", [True, False])
def test_a_dropped_plan_stays_until_its_step_has_run(named):
    before = tensors([5000, 77, 4097] * 40, "bf16", False)
    after = [copy_of(t) for t in before]
    busy = torch.zeros(1 << 30, dtype=torch.uint8, device=DEV), torch.zeros(1 << 30, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plan = fq.adamw_plan(after)
    table, nbytes = plan.device.data_ptr(), plan.device.numel()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(100):                     # the step waits for some 40 milliseconds
            busy[0].copy_(busy[1])
        if not named:
            fq.fq_adamw_step(plan, **HYPER)
    if named:
        fq.fq_adamw_step(plan, stream=side, **HYPER)
    del plan
    new = [torch.empty(nbytes, dtype=torch.uint8, device=DEV) for _ in range(8)]
    waiting = not side.query()
    assert waiting and table not in [t.data_ptr() for t in new]
    for t in new:
        t.fill_(0xFF)
    side.synchronize()
    torch.cuda.synchronize()
    check_f32(before, after)
