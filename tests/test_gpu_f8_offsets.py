"""GPU tests of lists of group offsets that are out of order or outside the
matrix, with every tile of the products: the kernels clamp them, so nothing
outside the outputs is written, nor any row of D that no group holds.  All
outputs lie inside larger buffers of a known pattern."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import f8_ref as R
from tests.test_gpu_f8 import SKINNY, TENSOR, _set, grouped_inputs, on_gpu

pytestmark = pytest.mark.gpu

BAD = [[0, 10, 5, 60], [-5, 20, 40, 60], [0, 20, 1000, 2000], [50, 40, 30, 20], [60, 0, 60, 0], [0, 60, 0, 60],
       [2 ** 31 - 1] * 4, [-2 ** 31] * 4, [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]]
MANY = [[0, 60] * 20 + [0], [60, 0] * 20 + [60]]   # forty groups, every other one with all rows
M, K, N, COLS = 60, 256, 140, 70
GUARD = 512


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


class Guarded:
    """A contiguous tensor between two guards."""

    def __init__(self, shape, dtype=torch.float32):
        n = 1
        for s in shape:
            n *= s
        self.raw = torch.full((n * dtype.itemsize + 2 * GUARD,), 0x55, dtype=torch.uint8, device="cuda")
        self.inside = self.raw[GUARD:-GUARD].view(dtype).view(*shape)

    def kept(self):
        return bool((self.raw[:GUARD] == 0x55).all()) and bool((self.raw[-GUARD:] == 0x55).all())


def held(offsets):
    """Rows that a clamped list gives to some group."""
    rows = set()
    for a, b in zip(offsets, offsets[1:]):
        lo = min(max(a, 0), M)
        rows |= set(range(lo, min(max(b, lo), M)))
    return rows


@pytest.mark.parametrize("cfg", [None] + SKINNY + TENSOR, ids=lambda c: "planned" if c is None else "-".join(str(v) for v in c.values()))
def test_rows_by_any_list(cfg):
    for bad in BAD + MANY:
        g = len(bad) - 1
        A, sa, Bt, sb, _, _ = grouped_inputs([0] * g, K, N, M, 81, B.GEMM_SCALE_BLOCKS)
        D = Guarded((M, N))
        plan = B.gemm_f8_grouped_plan(B.GEMM_GROUP_ROWS, g, M, K, N)
        if cfg:
            _set(**cfg)(plan)
        B.gemm_f8_grouped_run(plan, on_gpu(A), sa.cuda(), on_gpu(Bt), sb.cuda(),
                              torch.tensor(bad, dtype=torch.int32, device="cuda"), D.inside)
        torch.cuda.synchronize()
        assert D.kept(), bad
        out = [i for i in range(M) if i not in held(bad)]
        assert bool((D.inside.view(torch.uint8)[out] == 0x55).all()), bad


@pytest.mark.parametrize("cfg", [None] + SKINNY + TENSOR, ids=lambda c: "planned" if c is None else "-".join(str(v) for v in c.values()))
def test_quantised_columns_and_k_by_any_list(cfg):
    X = torch.randn(M, COLS, generator=R.gen(5)).cuda()
    for bad in BAD + MANY:
        g = len(bad) - 1
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kp = B.gemm_f8_padded_k(M, g)
        Q, S, W = Guarded((COLS, kp), R.E4M3), Guarded((kp // 128, COLS)), Guarded((g, COLS, COLS))
        B.gemm_f8_quantize_cols(X, Q.inside, S.inside, off)
        plan = B.gemm_f8_grouped_plan(B.GEMM_GROUP_K, g, COLS, kp, COLS, b_scale=B.GEMM_SCALE_ROWS)
        if cfg:
            _set(**cfg)(plan)
        B.gemm_f8_grouped_run(plan, Q.inside, S.inside, Q.inside, S.inside, off, W.inside)
        torch.cuda.synchronize()
        assert Q.kept() and S.kept() and W.kept(), bad
