"""GPU tests of the layer norm and its gradient with so many rows that every kernel
goes round its loop, and every slot of a ring is filled again, several times; and
that a row's NaN or infinity stays in its row where a kernel works on several rows
together.  Tolerances: as in test_gpu_layer_norm.py.  Sums over the rows are
tested with whole numbers below 2^24, which are exact in any order."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-5
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)]
# rows, d, pad.  On 152 SMs a team of the ring kernels takes 3 to 30 chunks of these through 2 to 8 slots.
CASES = [(40000, 384, 0), (30000, 1024, 0), (24000, 256, 0), (16000, 2048, 0), (5000, 8192, 0), (90000, 64, 0),
         (20919, 401, 0), (60000, 105, 0), (160000, 33, 0), (12000, 1001, 0), (5000, 4095, 0), (5000, 8191, 0),
         (20000, 500, 3), (40000, 24, 1)]


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


def nan(*shape):
    return torch.full(shape, float("nan"), device="cuda")


def normal(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("rows,d,pad", CASES)
def test_forward(rows, d, pad, tx, ty):
    g = generator(rows + d)
    # every row has a size of its own, so that another row's values are seen
    scale = 1 + torch.arange(rows, device="cuda")[:, None] % 97
    x, r = ((normal(g, rows, d) + 0.5) * scale).to(tx), normal(g, rows, d, dtype=tx)
    w, b = 1 + 0.2 * normal(g, d), 0.3 * normal(g, d)
    h, mean, var, rstd, y = R.layer_norm(x, r, w, b, EPS, tx)
    X, Rr = R.padded(x, pad)[0], R.padded(r, pad)[0]
    H, hbuf = R.padded(torch.zeros_like(x), pad, 0, 7.0)
    Y, ybuf = R.padded(torch.zeros(rows, d, dtype=ty, device="cuda"), pad, 0, 7.0)
    M, S = nan(rows), nan(rows)
    B.gemm_layer_norm(X, Rr, w, b, EPS, H, M, S, Y)
    assert torch.equal(H, h)
    off = 2.0 ** -18 * h.double().abs().mean(1)
    assert bool(((M.double() - mean).abs() <= off).all())
    rel = 2.0 ** -18 + off ** 2 / (2 * (var + EPS))
    assert bool(((S.double() - rstd).abs() <= rel * rstd).all())
    size = (h.double() - mean[:, None]).abs_() * rstd[:, None] * w.double().abs() + b.double().abs()
    size = (2.0 ** -17 + rel[:, None]) * size + (off * rstd)[:, None] * w.double().abs() * 1.01
    assert bool(((Y.double() - y).abs() <= size + R.HALF_STEP[ty] * (y.abs() + size)).all())
    for buf, view in ((hbuf, H), (ybuf, Y)):
        if pad:
            assert bool((R.outside(buf, view) == 7.0).all())


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("rows,d,pad", CASES)
def test_backward(rows, d, pad, tx, ty):
    g = generator(rows + d)
    scale = 1 + torch.arange(rows, device="cuda")[:, None] % 97
    x, w = (normal(g, rows, d) * scale).to(tx), 1 + 0.2 * normal(g, d)
    dy, dr = (normal(g, rows, d) * scale).to(ty), normal(g, rows, d, dtype=tx)
    mean, rstd = x.double().mean(1).float(), (1 / torch.sqrt(x.double().var(1, correction=0) + EPS)).float()
    dY, H, dR = R.padded(dy, pad)[0], R.padded(x, pad)[0], R.padded(dr, pad)[0]
    dX, buf = R.padded(torch.zeros_like(x), pad, 0, 7.0)
    dW, dB = nan(d), nan(d)
    B.gemm_layer_norm_backward(dY, H, w, mean, rstd, dR, dX, dW, dB)
    dx, _, _, size, _, _ = R.layer_norm_backward(dy, x, w, mean, rstd, dr)
    size = 2.0 ** -16 * size
    assert bool(((dX.double() - dx).abs() <= size + R.HALF_STEP[tx] * (dx.abs() + size)).all())
    if pad:
        assert bool((R.outside(buf, dX) == 7.0).all())
    # whole numbers, x = h and W = 0: dW, dbias and dX = dR are exact
    del dx, size
    x, dy = (torch.randint(-4, 5, (rows, d), generator=g, device="cuda").to(t) for t in (tx, ty))
    dY.copy_(dy)
    H.copy_(x)
    B.gemm_layer_norm_backward(dY, H, torch.zeros_like(w), torch.zeros_like(mean), torch.ones_like(rstd), dR, dX, dW, dB)
    assert torch.equal(dX, dR)
    assert torch.equal(dW.double(), (dy.double() * x.double()).sum(0)) and torch.equal(dB.double(), dy.double().sum(0))


@pytest.mark.parametrize("tx,ty", [(BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("rows,d,pad", CASES)
def test_a_bad_row_stays_alone(rows, d, pad, tx, ty):
    g = generator(d)
    x, r, dy = normal(g, rows, d, dtype=tx), normal(g, rows, d, dtype=tx), normal(g, rows, d, dtype=ty)
    w, b = 1 + 0.2 * normal(g, d), 0.3 * normal(g, d)
    bad = torch.tensor([0, 3, 50, 51, rows // 2, rows // 2 + 7, rows - 6, rows - 1], device="cuda")

    def run(x, dy):
        X, Rr, dY = R.padded(x, pad)[0], R.padded(r, pad)[0], R.padded(dy, pad)[0]
        H, Y = R.padded(torch.zeros_like(x), pad)[0], R.padded(torch.zeros_like(dy), pad)[0]
        dX, dW, dB = R.padded(torch.zeros_like(x), pad)[0], nan(d), nan(d)
        M, S = nan(rows), nan(rows)
        B.gemm_layer_norm(X, Rr, w, b, EPS, H, M, S, Y)
        B.gemm_layer_norm_backward(dY, H, w, M, S, Rr, dX, dW, dB)
        return H, M, S, Y, dX

    clean = run(x, dy)
    xb, dyb = x.clone(), dy.clone()
    for i, row in enumerate(bad.tolist()):
        at = (0, d - 1, d // 2, 1)[i % 4]
        xb[row, at] = float("nan") if i % 2 else float("inf")
    outs = run(xb, dy)
    good = torch.ones(rows, dtype=torch.bool, device="cuda")
    good[bad] = False
    for name, a, c in zip(("H", "mean", "rstd", "Y", "dX"), outs, clean):
        assert torch.equal(a[good], c[good]), name
    assert bool(outs[3][bad].isnan().all()) and bool(outs[4][bad].isnan().all())
    # the same for the gradient that comes in (an infinite dy makes mean(g) and mean(g xhat) infinite, so that every
    # dx of the row is an infinity or the NaN of two)
    for i, row in enumerate(bad.tolist()):
        dyb[row, (0, d - 1, d // 2, 1)[i % 4]] = float("nan") if i % 2 else float("inf")
    outs = run(x, dyb)
    assert torch.equal(outs[4][good], clean[4][good]) and not bool(outs[4][bad].isfinite().any())
