"""GPU tests of the layer norm (gemm_layer_norm) and its gradient
(gemm_layer_norm_backward), against 64-bit references.

Tolerances.  A row's sum is within 2^-18 of the sum of its magnitudes (each
thread adds at most 32 values, then a tree of at most ten steps: 42 2^-24), so
the mean is off by e <= 2^-18 mean|h|.  The squares of h - mean, off by e too,
sum to d (var + e^2) within 2^-18, so rstd is within
2^-18 + e^2 / (2 (var + eps)) of itself, and y within 2^-17 of the magnitudes
of its two terms plus e rstd |w| plus half a step of its type.  dX: 2^-16 of
the magnitudes of its terms plus half a step; dW, dbias: (rows + 64) 2^-24 of the sum of
the magnitudes."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-5
BF16, F32 = torch.bfloat16, torch.float32


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


def inputs(rows, d, seed, dtype, shift=0.5):
    g = R.gen(seed)
    spread = torch.exp(torch.randn(d, generator=g))
    x = (torch.randn(rows, d, generator=g) * spread + shift).to(dtype)
    r = (torch.randn(rows, d, generator=g) * 2).to(dtype)
    return x, r, 1.0 + 0.2 * torch.randn(d, generator=g), 0.3 * torch.randn(d, generator=g)


def check_forward(x, r, w, b, eps, tx, ty, pad=0, at=0, in_place=None):
    rows, d = x.shape
    h, mean, var, rstd, y = R.layer_norm(x, r, w, b, eps, tx)
    X = R.padded(x, pad, at)[0]
    Rr = None if r is None else R.padded(r, pad, at)[0]
    H, hbuf = R.padded(torch.zeros(rows, d, dtype=tx), pad, at, 7.0)
    if in_place is not None:
        H, hbuf = (X, None) if in_place == "x" else (Rr, None)
    Y, ybuf = R.padded(torch.zeros(rows, d, dtype=ty), pad, at, 7.0)
    M, S = torch.full((rows,), float("nan"), device="cuda"), torch.full((rows,), float("nan"), device="cuda")
    B.gemm_layer_norm(X, Rr, w.cuda(), None if b is None else b.cuda(), eps, H, M, S, Y)
    assert torch.equal(H.cpu(), h)
    off = 2.0 ** -18 * h.double().abs().mean(1)
    assert bool(((M.cpu().double() - mean).abs() <= off + 1e-40).all())
    rel = 2.0 ** -18 + off ** 2 / (2 * (var + eps))
    assert bool(((S.cpu().double() - rstd).abs() <= rel * rstd).all())
    term = ((h.double() - mean[:, None]) * rstd[:, None] * w.double()).abs()
    size = (2.0 ** -17 + rel[:, None]) * (term + (0 if b is None else b.double().abs())) + (off * rstd)[:, None] * w.double().abs() * 1.01
    err = (Y.cpu().double() - y).abs()
    assert bool((err <= size + R.HALF_STEP[ty] * (y.abs() + size) + 1e-40).all())
    for buf, view in ((hbuf, H), (ybuf, Y)):
        if buf is not None:
            assert bool((R.outside(buf, view) == 7.0).all())
    return Y


SHAPES = [(1, 1), (1, 8192), (3, 7), (5, 128), (2, 777), (700, 130), (9, 1000), (330, 1024), (400, 777), (2, 16384), (320, 8192),
          (3, 32768), (310, 20000), (2, 32761)]
TYPES = [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)]


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward(rows, d, tx, ty):
    x, r, w, b = inputs(rows, d, rows + d, tx)
    check_forward(x, r, w, b, EPS, tx, ty)
    check_forward(x, None, w, None, EPS, tx, ty)


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("d", [1, 8, 129, 256, 257, 512, 515, 768, 769])
def test_many_short_rows(d, tx, ty):
    x, r, w, b = inputs(1301, d, d, tx)
    check_forward(x, r, w, b, EPS, tx, ty)
    check_backward(1301, d, tx, ty)


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("pad,at", [(8, 0), (1, 0), (3, 1), (8, 4), (16, 8)])
@pytest.mark.parametrize("rows,d", [(5, 300), (330, 1024), (1300, 250), (160, 2056)])
def test_pitches_and_addresses(rows, d, pad, at, tx, ty):
    x, r, w, b = inputs(rows, d, rows + d, tx)
    check_forward(x, r, w, b, EPS, tx, ty, pad, at)
    check_forward(x, r, w, b, EPS, tx, ty, pad, at, "x")
    check_forward(x, r, w, b, EPS, tx, ty, pad, at, "r")
    check_backward(rows, d, tx, ty, pad, at)


def test_a_mean_far_from_zero():
    # one-pass variances lose everything here; the values' own spread is exact in fp32
    x = 4096.0 + (torch.arange(1024) % 16).float().repeat(8, 1)
    check_forward(x, None, torch.ones(1024), None, EPS, F32, F32)
    xb = (256.0 + 2 * (torch.arange(1024) % 16)).repeat(200, 1).to(BF16)
    check_forward(xb, None, torch.ones(1024), None, EPS, BF16, F32)


def test_constant_rows_and_special_values():
    rows, d = 6, 520
    x, _, w, b = inputs(rows, d, 1, F32)
    x[0], x[1] = 3.0, 0.0
    y = check_forward(x, None, w, b, EPS, F32, F32)
    assert torch.equal(y[0].cpu(), b) and torch.equal(y[1].cpu(), b)     # (h - mean) is zero
    x[2, 5], x[3, 7] = float("nan"), float("inf")
    Y, M, S = (torch.zeros(rows, d, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda"))
    B.gemm_layer_norm(x.cuda(), None, w.cuda(), b.cuda(), 0.0, None, M, S, Y)
    Y = Y.cpu()
    for row in (0, 1, 2, 3):      # eps = 0: 0 * infinity
        assert bool(Y[row].isnan().all())
    assert bool(Y[4:].isfinite().all())


def check_backward(rows, d, tx, ty, pad=0, at=0, seed=0):
    x, _, w, _ = inputs(rows, d, seed + rows + d, tx)
    dy, dr = R.normal((rows, d), seed + 1, 0.1, ty), R.normal((rows, d), seed + 2, 0.1, tx)
    _, mean, _, rstd, _ = R.layer_norm(x, None, w, None, EPS, tx)
    mean, rstd = mean.float(), rstd.float()
    W, M, S = w.cuda(), mean.cuda(), rstd.cuda()
    for use_dr in (True, False):
        dx, dw, db, size, sw, sb = R.layer_norm_backward(dy, x, w, mean, rstd, dr if use_dr else None)
        dY, H = R.padded(dy, pad, at)[0], R.padded(x, pad, at)[0]
        dR = R.padded(dr, pad, at)[0] if use_dr else None
        dX, buf = R.padded(torch.zeros(rows, d, dtype=tx), pad, at, 7.0)
        dW, dB = torch.full((d,), float("nan"), device="cuda"), torch.full((d,), float("nan"), device="cuda")
        B.gemm_layer_norm_backward(dY, H, W, M, S, dR, dX, dW, dB)
        err = (dX.cpu().double() - dx).abs()
        size = 2.0 ** -16 * size
        assert bool((err <= size + R.HALF_STEP[tx] * (dx.abs() + size) + 1e-40).all())
        part = (rows + 64) * 2.0 ** -24
        assert bool(((dW.cpu().double() - dw).abs() <= part * sw + 1e-30).all())
        assert bool(((dB.cpu().double() - db).abs() <= part * sb + 1e-30).all())
        assert bool((R.outside(buf, dX) == 7.0).all())
        # some outputs alone, with the same bits
        for ask_w, ask_b in ((True, False), (False, True), (False, False)):
            dX2 = R.padded(torch.zeros(rows, d, dtype=tx), pad, at, 7.0)[0]
            dW2, dB2 = torch.zeros_like(dW), torch.zeros_like(dB)
            B.gemm_layer_norm_backward(dY, H, W, M, S, dR, dX2, dW2 if ask_w else None, dB2 if ask_b else None)
            assert torch.equal(dX2, dX)
            assert not ask_w or torch.equal(dW2, dW)
            assert not ask_b or torch.equal(dB2, dB)
        if use_dr:        # in place of dR, and of dY
            B.gemm_layer_norm_backward(dY, H, W, M, S, dR, dR, dW2, dB2)
            assert torch.equal(dR, dX) and torch.equal(dW2, dW) and torch.equal(dB2, dB)
            if tx == ty:
                dR = R.padded(dr, pad, at)[0]
                B.gemm_layer_norm_backward(dY, H, W, M, S, dR, dY, dW2, dB2)
                assert torch.equal(dY, dX) and torch.equal(dW2, dW) and torch.equal(dB2, dB)


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("rows,d,pad,at", [
    (304, 401, 0, 0), (305, 401, 0, 0), (608, 511, 0, 0), (609, 511, 0, 0), (1216, 511, 0, 0), (1217, 500, 3, 1), (2433, 17, 0, 0),
    (4863, 192, 0, 0), (4865, 136, 0, 0),
    (4864, 512, 8, 0), (700, 16, 0, 0), (700, 16, 1, 1), (700, 9, 3, 1), (1000, 33, 15, 1), (613, 4088, 0, 0), (613, 4096, 8, 0), (613, 4104, 0, 0),
    (613, 4097, 0, 0), (620, 8184, 0, 0), (620, 8191, 0, 0), (620, 8192, 1, 0), (620, 8200, 0, 0), (620, 8193, 0, 0)])
def test_where_the_kernels_change(rows, d, pad, at, tx, ty):
    x, r, w, b = inputs(rows, d, rows + d, tx)
    check_forward(x, r, w, b, EPS, tx, ty, pad, at)
    check_backward(rows, d, tx, ty, pad, at)


@pytest.mark.parametrize("tx,ty", [(BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("rows,d", [(3, 40), (700, 40), (700, 136), (700, 1032), (700, 5000), (320, 9000)])
def test_matrices_that_lie_differently(rows, d, tx, ty):
    # every matrix with a pitch and an offset of its own: the same values as dense ones
    x, r, w, b = inputs(rows, d, rows + d, tx)
    dy, dr = R.normal((rows, d), 1, 0.1, ty), R.normal((rows, d), 2, 0.1, tx)
    _, mean, _, rstd, _ = R.layer_norm(x, r, w, b, EPS, tx)
    W, bias, M, S = w.cuda(), b.cuda(), mean.float().cuda(), rstd.float().cuda()
    mats = lambda *m: [R.padded(t, *m[i % len(m)], 7.0) for i, t in enumerate((x, r, x, dy, dy, dr, x))]  # noqa: E731
    outs = []
    for places in (((0, 0),), ((8, 0), (1, 1), (0, 0), (3, 2), (8, 8), (0, 0), (5, 3)), ((0, 0), (0, 0), (8, 0), (0, 1), (0, 0), (0, 1), (0, 0))):
        (X, _), (Rr, _), (H, hbuf), (Y, ybuf), (dY, _), (dR, _), (dX, xbuf) = mats(*places)
        dW, dB = torch.full((d,), float("nan"), device="cuda"), torch.full((d,), float("nan"), device="cuda")
        B.gemm_layer_norm(X, Rr, W, bias, EPS, H, torch.empty_like(M), torch.empty_like(S), Y)
        B.gemm_layer_norm_backward(dY, H, W, M, S, dR, dX, dW, dB)
        for buf, view in ((hbuf, H), (ybuf, Y), (xbuf, dX)):
            assert bool((R.outside(buf, view) == 7.0).all())
        outs.append((H, Y, dX, dW, dB))
    for other in outs[1:]:
        assert torch.equal(other[0], outs[0][0])
        # Sums may be taken in another order.  y and dx: each side is rounded once (half a step each), and the
        # sums behind them are off by a few 2^-24 of the row's size.  dw and db: each side by rows 2^-24 of the sum
        # of the terms' sizes, and |xhat| <= sqrt(d).
        step = 2 * R.HALF_STEP[tx]
        for got, want, eps in ((other[1], outs[0][1], 2.0 ** -7), (other[2], outs[0][2], max(step, 2.0 ** -12))):
            assert bool(((got.double() - want.double()).abs() <= eps * (want.double().abs() + 2.0 ** -10 * want.double().abs().max())).all())
        size = (rows + 64) * 2.0 ** -23 * dy.double().abs().sum(0).cuda()
        for got, want, most in ((other[3], outs[0][3], d ** 0.5), (other[4], outs[0][4], 1.0)):
            assert bool(((got.double() - want.double()).abs() <= most * size).all())


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES + [(5000, 64), (3000, 300), (200, 4104)])
def test_backward(rows, d, tx, ty):
    check_backward(rows, d, tx, ty)


def test_gradient_against_differences():
    rows, d = 3, 24
    x, _, w, b = inputs(rows, d, 1, F32)
    g = torch.randn(rows, d, generator=R.gen(2))
    Y, M, S = torch.zeros(rows, d, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    B.gemm_layer_norm(x.cuda(), None, w.cuda(), b.cuda(), EPS, None, M, S, Y)
    dX, dW, dB = torch.zeros(rows, d, device="cuda"), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")
    B.gemm_layer_norm_backward(g.cuda(), x.cuda(), w.cuda(), M, S, None, dX, dW, dB)

    def loss(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return (g.double() * (c / torch.sqrt(c.square().mean(1, keepdim=True) + EPS) * w + b)).sum()

    args = [x.double(), w.double(), b.double()]
    for i, got in enumerate((dX, dW, dB)):
        for at in range(0, args[i].numel(), 5):
            hi, lo = [a.clone() for a in args], [a.clone() for a in args]
            hi[i].view(-1)[at] += 1e-6
            lo[i].view(-1)[at] -= 1e-6
            want = (loss(*hi) - loss(*lo)) / 2e-6
            # differences of a sum of 72 terms in 64 bits: 1e-8 of it; the kernel: 2^-16 of its terms
            assert abs(got.cpu().double().view(-1)[at] - want) <= 1e-4 * (1 + abs(want))


def test_streams_and_graphs():
    rows, d = 700, 1032
    x, r, w, b = (t.cuda() for t in inputs(rows, d, 3, BF16))
    dy = R.normal((rows, d), 4, 0.1).cuda()

    def call(out):
        B.gemm_layer_norm(x, r, w, b, EPS, out["h"], out["m"], out["s"], out["y"])
        B.gemm_layer_norm_backward(dy, out["h"], w, out["m"], out["s"], None, out["dx"], out["dw"], out["db"])

    def outputs():
        e = lambda *s, t=F32: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
        return dict(h=e(rows, d, t=BF16), m=e(rows), s=e(rows), y=e(rows, d, t=BF16), dx=e(rows, d, t=BF16), dw=e(d), db=e(d))

    first = outputs()
    call(first)
    torch.cuda.synchronize()
    outs = [outputs() for _ in range(6)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        with torch.cuda.stream(streams[i % 3]):
            call(o)
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        o, graph = outputs(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(o)
        graphs.append((graph, o))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o in outs + [o for _, o in graphs]:
        for name, t in o.items():
            assert torch.equal(t, first[name]), name
