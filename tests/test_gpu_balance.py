"""GPU tests of the balance loss and the experts' counts (gemm_balance) and of
the gradient (gemm_balance_backward), against 64-bit references.

Tolerances.  With logits of magnitude at most x, the exponent of a probability
is off by at most (x + |lse|) 2^-24 beside exp's own 2^-22, and a row's sum of E terms by
(E / 32 + 6) 2^-24: p is within q = (2 x + 8) 2^-23 + (E / 32 + 8) 2^-24 of itself;
means over the rows add (rows / 32 + 200) 2^-24.  lse: q + 2^-23 |lse|.
Counts, offsets and used are exact."""

import math

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
COEF = 0.02


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


def forward(X, index, offsets=True, stream=None):
    rows, e = X.shape
    nan, i32 = float("nan"), dict(dtype=torch.int32, device="cuda")
    o = dict(counts=torch.full((e,), -7, **i32), offsets=torch.full((e + 1,), -7, **i32) if offsets else None,
             used=torch.full((1,), -7, **i32), lse=torch.full((rows,), nan, device="cuda"),
             probs=torch.full((e,), nan, device="cuda"), loss=torch.full((1,), nan, device="cuda"))
    B.gemm_balance(X, index, COEF, o["counts"], o["offsets"], o["used"], o["lse"], o["probs"], o["loss"], stream)
    return o


def check(x, index, pad=0, at=0, dtype=None):
    """Both passes of one case; returns the forward outputs."""
    rows, e = x.shape
    dtype = x.dtype
    counts, offsets, t, lse, probs, loss, p, f = R.balance(x, index, COEF)
    X = R.padded(x, pad, at)[0]
    o = forward(X, index.cuda())
    assert torch.equal(o["counts"].cpu().long(), counts) and torch.equal(o["offsets"].cpu().long(), offsets)
    assert int(o["used"]) == t
    finite = x.double()[x.isfinite()]
    most = finite.abs().max().item() if finite.numel() else 0.0
    q = (2 * most + 8) * 2.0 ** -23 + (e / 32 + 8) * 2.0 ** -24
    got = o["lse"].cpu().double()
    fin = lse.isfinite()
    assert torch.equal(got[~fin], lse[~fin])
    assert bool(((got - lse).abs()[fin] <= q + 2.0 ** -23 * lse.abs()[fin]).all())
    mean = q + (rows / 32 + 200) * 2.0 ** -24
    assert bool(((o["probs"].cpu().double() - probs).abs() <= mean * probs + 1e-38).all())
    assert abs(o["loss"].item() - loss.item()) <= (mean + (e / 32 + 12) * 2.0 ** -24) * loss.item()
    without = forward(X, index.cuda(), offsets=False)
    assert torch.equal(without["loss"], o["loss"]) and torch.equal(without["counts"], o["counts"])

    dloss = torch.tensor([1.5], device="cuda")
    for use_dr in (True, False):
        dr = R.normal((rows, e), 9, 0.01, dtype) if use_dr else None
        want, size = R.balance_gradient(p, f, t, COEF, 1.5, dr)
        dR = None if dr is None else R.padded(dr, pad, at)[0]
        dX, buf = R.padded(torch.zeros(rows, e, dtype=dtype), pad, at, 7.0)
        B.gemm_balance_backward(X, o["lse"], o["counts"], o["used"], COEF, dloss, dR, dX)
        err = (dX.cpu().double() - want).abs()
        size = (2 * q + (e / 32 + 12) * 2.0 ** -24 + lse.abs().where(fin, 0.0)[:, None] * 2.0 ** -23) * size
        assert bool((err <= size + R.HALF_STEP[dtype] * (want.abs() + size) + 1e-38).all())
        assert bool((R.outside(buf, dX) == 7.0).all())
        if use_dr:
            B.gemm_balance_backward(X, o["lse"], o["counts"], o["used"], COEF, dloss, dR, dR)
            assert torch.equal(dR, dX)
    return o


def routed(rows, e, k, seed, dtype, drop=0.05):
    x = R.normal((rows, e), seed, 2.0, dtype)
    index = x.float().topk(k, 1).indices.to(torch.int32)
    g = R.gen(seed + 1)
    index[torch.rand(rows, k, generator=g) < drop] = -1
    index[rows - rows // 8:] = -1
    return x, index.contiguous()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,e,k", [(1, 1, 1), (1, 8, 2), (48, 32, 2), (7, 5, 5), (100, 64, 8), (300, 33, 1), (1000, 130, 4),
                                      (40, 1024, 8), (5000, 16, 2), (3, 257, 3), (2500, 4, 1), (700, 600, 6), (20000, 3, 1)])
def test_balance(rows, e, k, dtype):
    x, index = routed(rows, e, k, rows + e, dtype)
    check(x, index)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("e", [7, 8, 60, 64, 256])
@pytest.mark.parametrize("pad,at", [(1, 0), (8, 0), (3, 1), (8, 4)])
def test_pitches_and_addresses(e, pad, at, dtype):
    x, index = routed(333, e, 2, e, dtype)
    check(x, index, pad, at)


def test_every_slot_empty_or_outside():
    x = R.normal((50, 24), 1, 1.0, F32)
    for value in (-1, 24, 2 ** 31 - 1, -2 ** 31):
        o = check(x, torch.full((50, 3), value, dtype=torch.int32))
        assert int(o["used"]) == 0 and o["loss"].item() == 0.0 and bool((o["probs"] == 0).all())
        assert bool((o["lse"] == math.inf).all())


def test_one_expert_takes_all_and_an_index_twice():
    x = R.normal((400, 12), 2, 1.0, F32)
    o = check(x, torch.full((400, 2), 5, dtype=torch.int32))
    assert o["counts"][5].item() == 800
    check(x, torch.tensor([[3, 3, -1]], dtype=torch.int32).repeat(400, 1))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masked_logits(dtype):
    x, index = routed(200, 40, 2, 3, dtype, drop=0.0)
    x[:, 30:] = -math.inf                                # experts that are switched off
    x[:, 29] = torch.finfo(dtype).min
    x[5] = -math.inf                                     # a row that its mask leaves nothing
    x[6] = torch.finfo(dtype).min                        # and one of the lowest value
    x[7], x[7, 3] = -math.inf, 2.0
    x[180:] = float("nan")                               # padding (see routed) is not read
    index[:175] = index[:175].clamp(max=28)
    keep = torch.cat([x[:175], x[180:]])
    kept = torch.cat([index[:175], index[180:]])
    clean = torch.where(keep.isnan(), torch.zeros_like(keep), keep)
    want = forward(clean.cuda(), kept.cuda())
    got = forward(keep.cuda(), kept.cuda())
    for name in want:
        assert torch.equal(want[name], got[name]), name
    counts, offsets, t, lse, probs, loss, p, f = R.balance(clean, kept, COEF)
    assert got["lse"][5].item() == -math.inf
    # of the experts that are switched off only row 6 is left, where all 40 are alike
    assert bool(((got["probs"][30:].cpu() * t * 40 - 1).abs() <= 2.0 ** -20).all())
    assert torch.equal(got["counts"].cpu().long(), counts) and int(got["used"]) == t
    assert bool(((got["probs"].cpu().double() - probs).abs() <= 2.0 ** -12 * probs + 1e-30).all())
    dX = torch.full(keep.shape, 3.0, dtype=dtype, device="cuda")
    B.gemm_balance_backward(keep.cuda(), got["lse"], got["counts"], got["used"], COEF, torch.ones(1, device="cuda"), None, dX)
    assert bool((dX[5] == 0).all()) and bool((dX[175:] == 0).all()) and bool((dX[7:175, 30:] == 0).all())
    assert bool(dX.isfinite().all())


def test_nan_and_infinity_in_a_used_row_are_seen():
    for bad in (float("nan"), math.inf):
        x, index = routed(60, 16, 2, 4, F32, drop=0.0)
        x[3, 2] = bad
        o = forward(x.cuda(), index.cuda())
        assert bool(o["loss"].isnan().all()) and bool(o["lse"][3].isnan())
        assert bool(o["lse"][:3].isfinite().all())
        dX = torch.zeros(60, 16, device="cuda")
        B.gemm_balance_backward(x.cuda(), o["lse"], o["counts"], o["used"], COEF, torch.ones(1, device="cuda"), None, dX)
        assert bool(dX[3].isnan().all()) and bool(dX[4:52].isfinite().all())


def test_gradient_against_differences():
    rows, e = 6, 5
    x, index = routed(rows, e, 2, 5, F32, drop=0.0)
    index[2] = -1
    o = forward(x.cuda(), index.cuda())
    dX = torch.zeros(rows, e, device="cuda")
    B.gemm_balance_backward(x.cuda(), o["lse"], o["counts"], o["used"], COEF, torch.ones(1, device="cuda"), None, dX)
    for i in range(rows):
        for j in range(e):
            hi, lo = x.double().clone(), x.double().clone()
            hi[i, j] += 1e-5
            lo[i, j] -= 1e-5
            want = (R.balance(hi, index, COEF)[5] - R.balance(lo, index, COEF)[5]) / 2e-5
            assert abs(dX[i, j].item() - want.item()) <= 1e-8 + 1e-4 * abs(want.item())


def test_offsets_feed_the_grouped_product():
    # the offsets of a top-1 router as gemm_f8_grouped_run takes them
    rows, e, k, n = 130, 6, 128, 128
    x, index = routed(rows, e, 1, 6, F32, drop=0.1)
    o = forward(x.cuda(), index.cuda())
    order = torch.argsort(torch.where(index[:, 0] < 0, e, index[:, 0]), stable=True)
    a = torch.randint(-4, 5, (rows, k), generator=R.gen(7)).float()
    w = torch.randint(-4, 5, (e, n, k), generator=R.gen(8)).float()
    D = torch.full((rows, n), 9.0, device="cuda")
    ones = torch.ones(1, rows, device="cuda")
    plan = B.gemm_f8_grouped_plan(B.GEMM_GROUP_ROWS, e, rows, k, n)
    B.gemm_f8_grouped_run(plan, a[order].cuda().to(torch.float8_e4m3fn), ones, w.cuda().to(torch.float8_e4m3fn),
                          torch.ones(e, 1, 1, device="cuda"), o["offsets"], D)
    D = D.cpu()
    for i, row in enumerate(order.tolist()):
        expert = int(index[row, 0])
        want = a[row] @ w[expert].T if expert >= 0 else torch.full((n,), 9.0)    # rows behind the last expert stay
        assert torch.equal(D[i], want)


def test_streams_and_graphs():
    x, index = routed(3000, 64, 4, 8, F32)
    X, I = x.cuda(), index.cuda()
    first = forward(X, I)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 3]):
            outs.append(forward(X, I))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = forward(X, I)
            o["dx"] = torch.empty_like(X)
            B.gemm_balance_backward(X, o["lse"], o["counts"], o["used"], COEF, o["loss"], None, o["dx"])
        graphs.append((graph, o))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o in outs + [o for _, o in graphs]:
        for name in first:
            assert torch.equal(o[name], first[name]), name
    assert torch.equal(graphs[0][1]["dx"], graphs[1][1]["dx"])
