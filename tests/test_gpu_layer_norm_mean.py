"""GPU tests of the layer norm's mean in each of its kernels: constant rows, whose
residual is exactly zero, and rows whose mean is far larger than their spread.

Constant rows.  A mean formed from a rounded sum is off by a few units in the
last place; the kernels take the mean of h - mean as a correction.  In a
constant row each h - mean is k units with k <= 22 and k^2 d < 2^24, so that the
correction is exact and y is the bias, to the bit (0 * rstd * w + bias); with
eps = 0 rstd is infinite and y NaN.  (Values to 1e22, so that k^2 d squared units
stay in range.)

Far means.  The first mean is off by at most 2^-18 mean|h|, the sums of
e = h - mean by 2^-18 of their magnitudes (42 additions in a row at most), and
adding the correction rounds once: the mean is within
2^-24 |mean| + 2^-18 mean|e| + 2^-36 mean|h|, u in short.  Before it, u alone was
2^-18 mean|h|.  var is within 2^-17 mean(e^2), so rstd within 2^-18 (1 + u^2 / var) + 2^-22
of itself, and y = (h - mean) rstd w + b within u rstd |w| and 2^-16 of its terms
beside its rounding."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-5
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)]
# rows, d, pad: few rows (a CTA each), warps, a warp per row, the ring, the unaligned kernel dense and with pitches, long rows
SHAPES = [(6, 776, 0), (6, 1001, 0), (3, 32749, 0), (1300, 24, 0), (1300, 120, 0), (1300, 200, 0), (2000, 640, 0), (700, 776, 0), (700, 1000, 0),
          (700, 7168, 0), (5000, 328, 0), (700, 1001, 0), (5000, 401, 0), (3000, 105, 0), (700, 500, 3), (700, 13, 1), (640, 9000, 0)]


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


def forward(x, w, b, eps, ty, pad, r=None):
    rows, d = x.shape
    X = R.padded(x, pad)[0]
    Rr, H = (None, None) if r is None else (R.padded(r, pad)[0], R.padded(torch.zeros_like(x), pad)[0])
    Y = R.padded(torch.zeros(rows, d, dtype=ty), pad)[0]
    M, S = torch.full((rows,), float("nan"), device="cuda"), torch.full((rows,), float("nan"), device="cuda")
    B.gemm_layer_norm(X, Rr, w, b, eps, H, M, S, Y)
    return M, S, Y


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("rows,d,pad", SHAPES)
def test_constant_rows(rows, d, pad, tx, ty):
    values = torch.tensor([3.0, 100.0, 1000.0, 1e4, 0.1, 1 / 3, -7.77e5, 1e-30, 1e22, 1 + 2.0 ** -23, -1.0, 0.0, 1.9999999, 1e-12])
    x = values[torch.arange(rows) % len(values)].to(tx)
    g = R.gen(d)
    w, b = (1 + 0.2 * torch.randn(d, generator=g)).cuda(), torch.randn(d, generator=g).cuda()
    for r in (None, torch.full((rows, d), 0.3).to(tx)):
        h = x if r is None else (x.float() + r[:, 0].float()).to(tx)
        M, S, Y = forward(x[:, None].repeat(1, d), w, b, EPS, ty, pad, r)
        assert torch.equal(M, h.float().cuda())
        assert bool(((S.double() - EPS ** -0.5).abs() <= 2.0 ** -22 * EPS ** -0.5).all())     # eps in fp32, a root, a division
        assert torch.equal(Y, b.to(ty).expand(rows, d))
        _, _, Y = forward(x[:, None].repeat(1, d), w, None, EPS, ty, pad, r)
        assert bool((Y == 0).all())
        M, S, Y = forward(x[:, None].repeat(1, d), w, b, 0.0, ty, pad, r)
        assert torch.equal(M, h.float().cuda()) and bool(S.isposinf().all()) and bool(Y.isnan().all())


@pytest.mark.parametrize("tx,ty", [(BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("rows,d,pad", SHAPES)
def test_means_far_from_zero(rows, d, pad, tx, ty):
    far, step = (256.0, 2.0) if tx == BF16 else (65536.0, 2.0 ** -5)      # multiples of the type's step there
    g = R.gen(rows + d)
    x = (far + step * torch.randint(0, 64 if tx == BF16 else 16, (rows, d), generator=g)).to(tx)
    w, b = 1 + 0.2 * torch.randn(d, generator=g), torch.randn(d, generator=g)
    M, S, Y = forward(x, w.cuda(), b.cuda(), EPS, ty, pad)
    h = x.double().cuda()
    mean = h.mean(1)
    e = h - mean[:, None]
    var = e.square().mean(1)
    rstd = 1 / torch.sqrt(var + EPS)
    u = 2.0 ** -24 * mean.abs() + 2.0 ** -18 * e.abs().mean(1) + 2.0 ** -36 * h.abs().mean(1)
    assert bool(((M.double() - mean).abs() <= u).all())
    rel = 2.0 ** -18 * (1 + u ** 2 / (var + EPS)) + 2.0 ** -22
    assert bool(((S.double() - rstd).abs() <= rel * rstd).all())
    term = e * rstd[:, None] * w.double().cuda()
    size = 2.0 ** -16 * (term.abs() + b.double().abs().cuda()) + (u * rstd)[:, None] * w.double().abs().cuda() * 1.01
    want = term + b.double().cuda()
    err = (Y.double() - want).abs()
    assert bool((err <= size + R.HALF_STEP[ty] * (want.abs() + size)).all())
