"""GPU tests of the RMS norm with the residual's addition and 8-bit output
(gemm_norm_f8, gemm_norm_i8) and of its gradient (gemm_norm_backward),
against 64-bit references.

Tolerances.  rstd: the mean of d squares in fp32 is within (d / 1024 + 40)
2^-24 of itself (each thread adds at most 32 squares or d / 1024 in a row,
then a tree), the division, root and reciprocal add four roundings; 2^-17 for
d <= 32768.  y = h * rstd * w is then within 2^-16, and so is a block's
scale.  An 8-bit value may differ by one step where y lies next to a rounding
boundary: the value it stands for is within half a step and 2^-16 of y (e4m3:
a step is 2^-3 of the value's binade, at least 2^-9 of the scale; int8: one
scale).  dX: 2^-16 of the sum of its terms' magnitudes plus half a unit of
its type; dW: rows * 2^-24 + 2^-17 of the sum of |dY xhat| over the rows."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import f8_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-6
REL = 2.0 ** -16
HALF_UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


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


def inputs(rows, d, seed, dtype):
    g = R.gen(seed)
    spread = torch.exp(torch.randn(d, generator=g))
    x = (torch.randn(rows, d, generator=g) * spread).to(dtype)
    r = (torch.randn(rows, d, generator=g) * 2).to(dtype)
    return x, r, 1.0 + 0.2 * torch.randn(d, generator=g)


def with_pitch(x, pad):
    buf = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device="cuda")
    buf[:, :x.shape[1]] = x.cuda()
    return buf[:, :x.shape[1]]


def bytes_out(rows, d, pad, dtype):
    buf = torch.full((rows, d + pad), 0x55, dtype=torch.uint8, device="cuda")
    return buf.view(dtype)[:, :d], buf


def check_f8(q, scale, y):
    rows, d = y.shape
    kb = (d + 127) // 128
    yp = torch.zeros(rows, kb * 128, dtype=torch.float64)
    yp[:, :d] = y
    want = torch.clamp_min(yp.view(rows, kb, 128).abs().amax(2) / 448.0, R.SCALE_MIN).T
    s = scale.cpu().double()
    assert bool(((s - want).abs() <= REL * want).all())
    full = R.expand_rows(scale.cpu(), d)
    v = q.cpu().float().double() * full
    code = (y / full).abs()
    step = torch.exp2(torch.floor(torch.log2(code.clamp_min(2.0 ** -6))) - 3)
    assert bool(((v - y).abs() <= (0.5 * step + REL * code) * full).all())


def check_i8(q, scale, y):
    want = torch.clamp_min(y.abs().amax(1) / 127.0, R.SCALE_MIN)
    s = scale.cpu().double()
    assert bool(((s - want).abs() <= REL * want).all())
    v = q.cpu().double() * s[:, None]
    assert bool(((v - y).abs() <= 0.5 * s[:, None] + REL * y.abs()).all())
    assert int(q.min()) >= -127


SHAPES = [(1, 1), (1, 8192), (3, 7), (5, 128), (2, 777), (700, 130), (9, 1000), (330, 1024), (400, 777), (2, 16384),
          (320, 8192), (3, 32768), (310, 20000), (2, 32761)]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_norm_forward(rows, d, dtype, residual):
    x, r, w = inputs(rows, d, rows + d, dtype)
    h, rstd, y = R.norm(x, r if residual else None, w, EPS, dtype)
    X, Rr, W = x.cuda(), r.cuda() if residual else None, w.cuda()
    for to_i8 in (False, True):
        H, S1 = torch.empty(rows, d, dtype=dtype, device="cuda"), torch.empty(rows, device="cuda")
        Q, buf = bytes_out(rows, d, 0, torch.int8 if to_i8 else R.E4M3)
        S = torch.empty(rows if to_i8 else ((d + 127) // 128, rows), device="cuda")
        (B.gemm_norm_i8 if to_i8 else B.gemm_norm_f8)(X, Rr, W, EPS, H, S1, Q, S)
        torch.cuda.synchronize()
        assert torch.equal(H.cpu(), h)
        assert bool(((S1.cpu().double() - rstd).abs() <= 2.0 ** -17 * rstd).all())
        (check_i8 if to_i8 else check_f8)(Q, S, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1, 8, 129, 256, 257, 512, 515, 768, 769])
def test_norm_many_short_rows(d, dtype):
    # a warp per row up to 768 elements; the last CTA has fewer rows than warps
    test_norm_forward(1301, d, dtype, True)
    test_norm_backward(1301, d, dtype, True)


@pytest.mark.parametrize("rows,d", [(1301, 300), (1216, 256)])
def test_norm_short_rows_in_place(rows, d):
    test_norm_pitches_and_in_place(rows, d, torch.bfloat16)


def test_norm_short_rows_special():
    # a row of zeros, and a NaN and an infinity that stay in their rows
    rows, d = 1301, 300
    x, r, w = inputs(rows, d, 31, torch.bfloat16)
    h, rstd, y = R.norm(x, r, w, EPS, torch.bfloat16)
    bad = [4, 9, 1300]
    x[bad[0]], r[bad[0]] = 0, 0
    x[bad[1], 7], x[bad[2], 299] = float("nan"), float("inf")
    keep = torch.ones(rows, dtype=torch.bool)
    keep[bad] = False
    Q, S = torch.empty(rows, d, dtype=R.E4M3, device="cuda"), torch.empty(3, rows, device="cuda")
    B.gemm_norm_f8(x.cuda(), r.cuda(), w.cuda(), EPS, torch.empty_like(x).cuda(), None, Q, S)
    check_f8(Q[keep.cuda()].contiguous(), S[:, keep.cuda()].contiguous(), y[keep])
    assert bool((Q[bad[0]].float() == 0).all()) and bool(torch.isnan(Q[bad[1]].float()).any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(3, 777), (400, 256)])
def test_norm_pitches_and_in_place(rows, d, dtype):
    x, r, w = inputs(rows, d, 5, dtype)
    h, _, y = R.norm(x, r, w, EPS, dtype)
    for pads in ((0, 0, 0, 0), (8, 16, 24, 8), (1, 2, 3, 5), (8, 8, 8, 3)):
        X, Rr = with_pitch(x, pads[0]), with_pitch(r, pads[1])
        H, Q = with_pitch(torch.zeros_like(x), pads[2]), bytes_out(rows, d, pads[3], R.E4M3)
        S = torch.empty((d + 127) // 128, rows, device="cuda")
        B.gemm_norm_f8(X, Rr, w.cuda(), EPS, H, None, Q[0], S)
        assert torch.equal(H.cpu(), h) and bool((Q[1][:, d:] == 0x55).all())
        check_f8(Q[0].contiguous(), S, y)
        # the residual stream updated in place, over R and over X
        B.gemm_norm_f8(X, Rr, w.cuda(), EPS, Rr, None, Q[0], S)
        assert torch.equal(Rr.cpu(), h)
        Rr = with_pitch(r, pads[1])
        B.gemm_norm_f8(X, Rr, w.cuda(), EPS, X, None, Q[0], S)
        assert torch.equal(X.cpu(), h)
        check_f8(Q[0].contiguous(), S, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [6144, 6145, 8191, 12288])
def test_norm_many_long_rows(d, dtype):
    test_norm_forward(310, d, dtype, True)


def test_norm_special_rows():
    rows, d = 6, 300
    x, _, w = inputs(rows, d, 9, torch.float32)
    x[1], x[2, 5], x[3, 7], x[4] = 0.0, float("inf"), float("nan"), 1e-30
    Q, S = bytes_out(rows, d, 0, R.E4M3)[0], torch.empty(3, rows, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    B.gemm_norm_f8(x.cuda(), None, w.cuda(), EPS, None, rstd, Q, S)
    q, s = Q.cpu().view(torch.uint8), S.cpu()
    assert bool((q[1] == 0).all()) and bool((s[:, 1] == R.SCALE_MIN).all())
    assert q[2, 5].item() & 0x7F == 0x7F and bool((q[3] & 0x7F == 0x7F).all())
    for i in (0, 4, 5):
        _, _, y = R.norm(x[i:i + 1], None, w, EPS, torch.float32)
        check_f8(Q[i:i + 1].contiguous(), S[:, i:i + 1].contiguous(), y)
    Q8, S8 = bytes_out(rows, d, 0, torch.int8)[0], torch.empty(rows, device="cuda")
    B.gemm_norm_i8(x.cuda(), None, w.cuda(), EPS, None, None, Q8, S8)
    assert bool(S8[2].isnan()) and bool(S8[3].isnan()) and bool((Q8[1] == 0).all())
    assert bool(S8[[0, 1, 4, 5]].isfinite().all())


def test_norm_int8_feeds_the_requantised_product():
    m, k, n = 150, 320, 200
    x, r, w = inputs(m, k, 11, torch.bfloat16)
    wt = torch.randint(-127, 128, (n, k), generator=R.gen(3), dtype=torch.int8)
    cs = torch.rand(n, generator=R.gen(4)) / 1000 + 1e-4
    Q, S = torch.empty(m, k, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    H, D = torch.empty(m, k, dtype=torch.bfloat16, device="cuda"), torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    B.gemm_norm_i8(x.cuda(), r.cuda(), w.cuda(), EPS, H, None, Q, S)
    B.gemm_i8_run_requant(B.gemm_i8_plan(m, k, n), Q, wt.cuda(), S, cs.cuda(), D)
    c = Q.cpu().double() @ wt.double().T * S.cpu().double()[:, None] * cs.double()
    assert bool(((D.cpu().double() - c).abs() <= 1.01 * 2.0 ** -8 * c.abs()).all())


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_norm_backward(rows, d, dtype, residual):
    h, dr, w = inputs(rows, d, rows + 3 * d, dtype)
    dy = torch.randn(rows, d, generator=R.gen(d)).to(dtype)
    _, rstd, _ = R.norm(h, None, w, EPS, dtype)
    rstd = rstd.float()
    dx, dw = R.norm_backward(dy, h, w, rstd, dr if residual else None)
    dX, dW = torch.empty(rows, d, dtype=dtype, device="cuda"), torch.full((d,), 7.0, device="cuda")
    args = (dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dr.cuda() if residual else None)
    B.gemm_norm_backward(*args, dX, dW)
    torch.cuda.synchronize()
    xhat, g = h.double() * rstd.double()[:, None], dy.double() * w.double()
    terms = rstd.double()[:, None] * (g.abs() + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    terms = terms + (dr.double().abs() if residual else 0.0)
    assert bool(((dX.cpu().double() - dx).abs() <= REL * terms + HALF_UNIT[dtype] * dx.abs()).all())
    S = (dy.double() * xhat).abs().sum(0)
    assert bool(((dW.cpu().double() - dw).abs() <= (rows * 2.0 ** -24 + 2.0 ** -17) * S).all())
    # the same bits again, and without dW
    dX2, dW2 = torch.empty_like(dX), torch.empty_like(dW)
    B.gemm_norm_backward(*args, dX2, dW2)
    assert torch.equal(dX2, dX) and torch.equal(dW2, dW)
    B.gemm_norm_backward(*args, dX2.zero_(), None)
    assert torch.equal(dX2, dX)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [12032, 12033, 12288, 12289])
def test_norm_backward_around_48_kib_of_sums(d, dtype):
    # dw's sums of one CTA take 48 KiB at 12288 columns, what a kernel has without asking for more
    test_norm_backward(5, d, dtype, True)
    test_norm_backward(160, d, dtype, False)


def test_norm_backward_in_place_and_pitches():
    rows, d = 350, 300
    h, dr, w = inputs(rows, d, 21, torch.bfloat16)
    dy = torch.randn(rows, d, generator=R.gen(22)).to(torch.bfloat16)
    rstd = R.norm(h, None, w, EPS, torch.bfloat16)[1].float()
    want = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    want_w = torch.empty(d, device="cuda")
    B.gemm_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dr.cuda(), want, want_w)
    for pads in ((4, 8, 12), (1, 3, 5)):
        DR, dW = with_pitch(dr, pads[2]), torch.empty(d, device="cuda")
        B.gemm_norm_backward(with_pitch(dy, pads[0]), with_pitch(h, pads[1]), w.cuda(), rstd.cuda(), DR, DR, dW)
        assert torch.equal(DR, want) and torch.equal(dW, want_w)


def test_norm_gradient_against_differences():
    """dX and dW against central differences of the 64-bit forward, for the
    loss sum(dy * y): step e, error O(e^2) times third derivatives (below
    1e-7 here) and 1e-10 of rounding."""
    rows, d, e = 3, 40, 1e-3
    h, _, w = inputs(rows, d, 31, torch.float32)
    dy = torch.randn(rows, d, generator=R.gen(32))

    def loss(hh, ww):
        rstd = 1.0 / torch.sqrt(hh.square().mean(1) + EPS)
        return (dy.double() * hh * rstd[:, None] * ww).sum()

    rstd = (1.0 / torch.sqrt(h.double().square().mean(1) + EPS)).float()
    dX, dW = torch.empty(rows, d, device="cuda"), torch.empty(d, device="cuda")
    B.gemm_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), None, dX, dW)
    H, W = h.double(), w.double()
    for i, j in [(0, 0), (1, 7), (2, 39), (0, 20)]:
        p = torch.zeros_like(H)
        p[i, j] = e
        num = (loss(H + p, W) - loss(H - p, W)) / (2 * e)
        assert abs(dX[i, j].item() - num.item()) <= 2e-5 * float(dy.abs().max())
        p = torch.zeros_like(W)
        p[j] = e
        num = (loss(H, W + p) - loss(H, W - p)) / (2 * e)
        assert abs(dW[j].item() - num.item()) <= 2e-5 * float(dy.abs().sum())
