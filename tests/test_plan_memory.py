"""Where an AdamW plan's two copies lie and how long: shown with a stand-in for
the device's memory, without a device."""
import os
from types import SimpleNamespace

import pytest

import fp4_block_quantization_fq_amd as fq


@pytest.fixture(autouse=True)
def built():
    if not os.path.exists(fq.LIB_PATH):
        pytest.skip("libfq.so not built")


def test_the_table_belongs_to_every_stream_that_reads_it():
    """A step on another stream than the plan was made on marks the table's memory
    as used there before it launches, once for each stream."""
    marked, asked = [], []
    plan = fq.adamw_plan([])
    one, two = SimpleNamespace(cuda_stream=0x100), SimpleNamespace(cuda_stream=0x200)
    plan.device = SimpleNamespace(record_stream=lambda s: marked.append(s.cuda_stream))
    for s in (one, one, two):
        plan._read_on(s)
    assert marked == [0x100, 0x200]
    # an empty plan's step launches nothing, and asks all the same
    plan.device, plan._read_on = None, lambda s: asked.append(s.cuda_stream)
    for s in (one, two, SimpleNamespace(cuda_stream=plan.stream)):
        fq.fq_adamw_step(plan, lr=1e-3, step=1, stream=s)
    assert asked == [0x100, 0x200]


def test_the_host_copy_is_in_host_memory():
    """Whatever device torch makes tensors on by default: the library writes the
    copy with plain stores."""
    import torch
    for kind in ("meta", "cpu"):
        with torch.device(kind):
            plan = fq.adamw_plan([])
        assert plan.host.device.type == "cpu"
        fq.fq_adamw_step(plan, lr=1e-3, step=1, stream=SimpleNamespace(cuda_stream=0))
