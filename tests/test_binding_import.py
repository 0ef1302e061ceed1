"""The row operators' extension in a process that has not imported torch."""
import os
import subprocess
import sys

import pytest

import fp4_block_quantization_fq_amd as fq


def test_a_call_that_meets_no_tensor_still_names_it():
    if not os.path.exists(fq.LIB_PATH):
        pytest.skip("libfq.so not built")
    code = ("import fp4_block_quantization_fq_amd as fq\n"
            "try:\n    fq.fq_rmsnorm_fwd([[1.0]], [1.0], 1e-5, y=1)\n"
            "except TypeError as e:\n    print(e)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(fq.__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert "x must be a tensor, not list" in out.stdout, out.stderr
