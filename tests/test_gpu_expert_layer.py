"""The example's training step on the 8-bit operators against the same layer
in fp32 torch.  e4m3 keeps three fraction bits: a value is off by 2^-4 at
most, by 2^-4 / sqrt(3) = 3.6 % rms at worst.  A result that has passed
through q such roundings of one of the factors each is off by about sqrt(q) 3.6 %;
the longest chain here (dw1: the normed row, the hidden gradient's two
products and their weights) has seven, 9.5 %; the activation's slope adds to
it, so 15 % is allowed, and rows of a wrong expert would give 100 %."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("rows,d,ff,experts", [(1000, 512, 768, 6), (37, 256, 200, 16), (1, 128, 130, 3)])
def test_expert_layer_step(rows, d, ff, experts):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_int8_matrix_gb300 import binding as B
    from dense_int8_matrix_gb300 import build
    build.build()
    import expert_layer
    errors = expert_layer.compare(rows, d, ff, experts)
    assert all(e < 0.15 for e in errors.values()), errors
    st, code = B.gemm_device_error()
    assert st == B.GEMM_OK, "device error word set: code %d" % code
