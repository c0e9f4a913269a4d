"""GPU test of the sums behind bfloat16 outputs.  All operands are positive, where
the tensor core's truncation always points one way.

An MMA adds 16 products and truncates: at most 2^-23 of the running sum.  Over
a chunk of c of them the running sum grows evenly, so that the chunk is short by
(c + 1) / 2 * 2^-23 of itself at most, and so are the sums of the chunks, which are
rounded to nearest: c = 32 (512 products) in the small tiles, 16.5 units of 2^-23;
in the two-SM tiles 96 in the first chunk and 64 in the others, of 8192 products
48.5 * 1536 / 8192 + 32.5 * 6656 / 8192 = 35.5.  The mean of (D - the exact value's rounding) is that shortfall: outputs
that are rounded otherwise for it differ by a step, 2^-7 of the value at most, and
are a share of p < 2^-9 of the N outputs, which makes the mean uncertain by 4 2^-7 sqrt(p / N)
(four standard deviations)."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_int8_matrix_gb300 import build
    build.build()
    B.load()
    yield
    st, code = B.gemm_device_error()
    assert st == B.GEMM_OK, "device error word set: code %d" % code


@pytest.mark.parametrize("path,bm,bn,split,units", [(B.GEMM_PATH_SKINNY, 16, 128, 1, 16.5), (B.GEMM_PATH_SKINNY, 32, 128, 1, 16.5),
                                                   (B.GEMM_PATH_SKINNY, 64, 128, 2, 16.5), (B.GEMM_PATH_SKINNY, 128, 128, 1, 16.5),
                                                   (B.GEMM_PATH_TENSOR, 256, 256, 1, 35.5), (B.GEMM_PATH_TENSOR, 256, 128, 1, 35.5)])
def test_shortfall_of_positive_sums(path, bm, bn, split, units):
    m, k, n = 512, 8192, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    a = torch.randn(m, k, generator=g, device="cuda").abs().to(torch.bfloat16)
    w = torch.randn(n, k, generator=g, device="cuda").abs().to(torch.bfloat16)
    plan = B.gemm_bf16_linear_plan(m, k, n)
    plan.path, plan.bm, plan.bn, plan.split_k = path, bm, bn, split
    D = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.gemm_bf16_linear_run(plan, a, w, D)
    exact = a.double() @ w.double().T
    short = -((D.double() - exact.to(torch.bfloat16).double()) / exact).mean().item()
    noise = 4 * 2.0 ** -7 * (2.0 ** -9 / (m * n)) ** 0.5
    assert -noise <= short <= units * 2.0 ** -23 + noise
