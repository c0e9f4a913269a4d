"""The trace counts every kernel that the 8-bit operators launch."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import f8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_int8_matrix_gb300 import build
    build.build()
    B.load()


def counted(call):
    B.gemm_trace_begin(16, 1)
    call()
    torch.cuda.synchronize()
    _, timed, launches = B.gemm_trace_collect()
    return timed, launches


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d,want", [(400, 512, 2), (20, 512, 2), (1, 512, 1)])
def test_norm_backward_counts_the_reduction_of_dw(rows, d, want, dtype):
    # the CTAs' sums of dw are added by a second kernel, unless one CTA has all rows
    x = torch.randn(rows, d, device="cuda").to(dtype)
    w, rstd, dx = torch.ones(d, device="cuda"), torch.ones(rows, device="cuda"), torch.empty_like(x)
    dw = torch.empty(d, device="cuda")
    for out, n in ((dw, want), (None, 1)):
        timed, launches = counted(lambda: B.gemm_norm_backward(x, x, w, rstd, None, dx, out))
        assert launches == [n if k == B.GEMM_KERNEL_STAGE else 0 for k in range(B.GEMM_KERNEL_KINDS)]
        assert timed[B.GEMM_KERNEL_STAGE] == 1


def test_the_other_calls_count_one():
    x = torch.randn(40, 256, device="cuda")
    q, s = torch.empty(40, 256, dtype=R.E4M3, device="cuda"), torch.empty(2, 40, device="cuda")
    one = lambda kind: [1 if k == kind else 0 for k in range(B.GEMM_KERNEL_KINDS)]  # noqa: E731
    assert counted(lambda: B.gemm_f8_quantize(x, q, s))[1] == one(B.GEMM_KERNEL_STAGE)
    assert counted(lambda: B.gemm_norm_f8(x, None, torch.ones(256, device="cuda"), 1e-6, None, None, q, s))[1] == one(
        B.GEMM_KERNEL_STAGE)
    plan = B.gemm_f8_plan(40, 256, 40, b_scale=B.GEMM_SCALE_ROWS)
    kind = B.GEMM_KERNEL_SKINNY if plan.path == B.GEMM_PATH_SKINNY else B.GEMM_KERNEL_TC
    assert counted(lambda: B.gemm_f8_run(plan, q, s, q, s, torch.empty(40, 40, device="cuda")))[1] == one(kind)
