"""GPU tests of the int8 norm (gemm_norm_i8) where y = h * rstd * W is NaN
although the row's mean square is finite: a NaN in W, an infinite W where h is
0, and a row of zeros at eps = 0 (rstd is infinite).  int8 holds no NaN, so the
row's scale has to carry it into the product that reads the row.  Both forms of
the kernel are run: a warp per row (many short rows) and a CTA per row."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import f8_ref as R
from tests.test_gpu_norm import EPS, check_i8, inputs

pytestmark = pytest.mark.gpu

# a warp per row; a CTA per row with one, two and four vectors per thread, aligned rows and others
SHAPES = [(1301, 300), (1301, 512), (6, 300), (9, 1), (320, 1000), (400, 2048), (310, 6152), (2, 32761)]


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


def run(x, w, eps, r=None):
    rows, d = x.shape
    Q, S = torch.full((rows, d), 99, dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda")
    H = None if r is None else torch.empty(rows, d, dtype=x.dtype, device="cuda")
    B.gemm_norm_i8(x.cuda(), None if r is None else r.cuda(), w.cuda(), eps, H, None, Q, S)
    return Q, S


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_nan_in_w(rows, d, dtype):
    x, r, w = inputs(rows, d, 7 * rows + d, dtype)
    w[d // 2] = float("nan")
    for res in (None, r):
        Q, S = run(x, w, EPS, res)
        assert bool(S.isnan().all()), "%d of %d rows have a finite scale" % (int((~S.isnan()).sum()), rows)
        assert bool((Q == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [s for s in SHAPES if s[1] > 1])
def test_infinite_w_where_h_is_zero(rows, d, dtype):
    # rows whose h is 0 in the column of the infinite weight are NaN there;
    # the others are infinite there, and the product that reads them is NaN too
    x, _, w = inputs(rows, d, 11 * rows + d, dtype)
    j = d - 1
    w[j] = float("inf")
    x[:, j] = 1.0
    x[::2, j] = 0.0
    Q, S = run(x, w, EPS)
    assert bool(S[::2].isnan().all())
    assert not bool(S.isfinite().any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_row_of_zeros_without_eps(rows, d, dtype):
    x, _, w = inputs(rows, d, 13 * rows + d, dtype)
    zero = [0, rows - 1]
    x[zero] = 0.0
    keep = torch.ones(rows, dtype=torch.bool)
    keep[zero] = False
    _, _, y = R.norm(x, None, w, 0.0, dtype)
    Q, S = run(x, w, 0.0)
    assert bool(S[zero].isnan().all())
    if bool(keep.any()):
        check_i8(Q[keep.cuda()], S[keep.cuda()], y[keep])
    # with an eps a row of zeros is zero
    Q, S = run(x, w, EPS)
    assert bool((Q[zero] == 0).all()) and bool((S[zero] == R.SCALE_MIN).all())


def test_nan_reaches_the_requantised_product():
    m, k, n = 40, 320, 96
    x, _, w = inputs(m, k, 3, torch.bfloat16)
    w[17] = float("nan")
    Q, S = run(x, w, EPS)
    wt = torch.randint(-127, 128, (n, k), generator=R.gen(3), dtype=torch.int8)
    D = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    B.gemm_i8_run_requant(B.gemm_i8_plan(m, k, n), Q, wt.cuda(), S, torch.ones(n, device="cuda"), D)
    assert bool(D.isnan().all())
