"""GPU tests of the bfloat16 product with bias, activation and residual
(gemm_bf16_linear_run) and of the activation's gradient
(gemm_activation_backward), against 64-bit references.

Tolerances.  A product of bfloat16 values is exact in fp32; sums of k of them
are within k 2^-23 of the sum of their magnitudes S (one truncation of at most
2^-23 of a partial sum for each), and whole numbers whose sums stay below 2^24
are exact, so with those every output must be the rounded exact value.  The
activations and their slopes are smooth with a slope of at most 1.2 and are
themselves within 2^-19 of max(1, |v|): exp is within (2 + 1.16 |x|) 2^-23 of
itself, and x^2 exp(-x) stays below 0.6.  An output is off by half a step of its type more.
Column sums of r rows: r 2^-24 of the sum of the magnitudes."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

NT, NN, TN = B.GEMM_FORM_NT, B.GEMM_FORM_NN, B.GEMM_FORM_TN
GRAD = B.GEMM_ACT_GRADIENT
ACT_ERR = 2.0 ** -19


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


def plans(form, m, k, n):
    """The plan's own choice and every other configuration."""
    def edit(**kw):
        p = B.gemm_bf16_linear_plan(m, k, n, form)
        for name, value in kw.items():
            setattr(p, name, value)
        return p

    yield edit()
    for bn in (128, 256):
        yield edit(path=B.GEMM_PATH_TENSOR, bm=256, bn=bn, split_k=1)
    for bm in (64, 128) if form == TN else (16, 32, 64, 128):
        for split in (1, 2, 4, 8):
            yield edit(path=B.GEMM_PATH_SKINNY, bm=bm, bn=128, split_k=split)


def filled(*shape, dtype=torch.bfloat16, fill=float("nan")):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


SHAPES = [(1, 1, 1), (1, 64, 8), (1, 8192, 300), (3, 7, 5), (16, 128, 128), (17, 777, 129), (100, 1000, 333), (128, 64, 256),
          (257, 65, 255), (300, 640, 520), (513, 129, 1000), (40, 2050, 2049)]


@pytest.mark.parametrize("form", [NT, NN, TN])
@pytest.mark.parametrize("m,k,n", SHAPES)
def test_whole_numbers_are_exact(form, m, k, n):
    A, Bm, a, b = R.operands(form, m, k, n, R.whole)
    want = a @ b
    for plan in plans(form, m, k, n):
        for dtype in (torch.float32, torch.bfloat16):
            D = filled(m, n, dtype=dtype)
            B.gemm_bf16_linear_run(plan, A.cuda(), Bm.cuda(), D)
            assert torch.equal(D.cpu(), want.to(dtype)), (plan.as_dict(), dtype)


@pytest.mark.parametrize("form", [NT, NN, TN])
def test_whole_numbers_of_a_large_product(form):
    m, k, n = 1100, 2088, 2304   # several rounds of tiles with halves; every operand's pitch is aligned
    A, Bm, a, b = R.operands(form, m, k, n, R.whole)
    want = (a.cuda() @ b.cuda())
    for plan in plans(form, m, k, n):
        D = filled(m, n, dtype=torch.float32)
        B.gemm_bf16_linear_run(plan, A.cuda(), Bm.cuda(), D)
        assert torch.equal(D.double(), want), plan.as_dict()


def check(got, want, size, dtype):
    """got against want whose error before the last rounding is at most size."""
    err = (got.cpu().double() - want).abs()
    limit = size + R.HALF_STEP[dtype] * (want.abs() + size) + 2.0 ** -126
    assert bool((err <= limit).all()), "off by up to %g of the limit" % (err / limit).max().item()


@pytest.mark.parametrize("act", list(R.ACTS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k,n", [(1, 1000, 264), (5, 77, 131), (150, 320, 264), (300, 96, 700)])
def test_epilogue(act, dtype, m, k, n):
    A, Bm, a, b = R.operands(NT, m, k, n, lambda s, seed: R.normal(s, seed, 2.0 if seed == 1 else k ** -0.5))
    bias = torch.randn(n, generator=R.gen(3))
    res, z_in = R.normal((m, n), 4, 3.0, dtype), R.normal((m, n), 5, 2.0)
    v = a @ b + bias.double()
    S = k * 2.0 ** -23 * (a.abs() @ b.abs()) + 2.0 ** -23 * (v.abs() + bias.double().abs())
    dA, dB, dbias, dres, dz = A.cuda(), Bm.cuda(), bias.cuda(), res.cuda(), z_in.cuda()
    for plan in plans(NT, m, k, n):
        for use_bias in (True, False):
            for use_res in (True, False):
                vv = v if use_bias else a @ b
                rr = res.double() if use_res else torch.zeros(m, n, dtype=torch.float64)
                D, Z = filled(m, n, dtype=dtype), filled(m, n)
                B.gemm_bf16_linear_run(plan, dA, dB, D, bias=dbias if use_bias else None, activation=R.ACTS[act], Z=Z,
                                       residual=dres if use_res else None)
                size = 1.2 * S + ACT_ERR * vv.abs().clamp(min=1) + 2.0 ** -24 * rr.abs()
                check(D, R.act(act, vv) + rr, size, dtype)
                check(Z, vv, S, torch.bfloat16)
        # the gradient form: Z is read, and left as it is
        D, Z = filled(m, n, dtype=dtype), dz.clone()
        B.gemm_bf16_linear_run(plan, dA, dB, D, bias=dbias, activation=R.ACTS[act] | GRAD, Z=Z, residual=dres)
        s = R.slope(act, z_in)
        check(D, v * s + res.double(), S * s.abs() + 2 * ACT_ERR * v.abs() + 2.0 ** -24 * res.double().abs(), dtype)
        assert torch.equal(Z, dz)


@pytest.mark.parametrize("form", [NT, NN, TN])
@pytest.mark.parametrize("pad,at", [(0, 0), (8, 0), (1, 0), (3, 1), (8, 4), (24, 8)])
def test_pitches_and_addresses(form, pad, at):
    m, k, n = 70, 200, 136
    A, Bm, a, b = R.operands(form, m, k, n, R.whole)
    res = R.whole((m, n), 3)
    want = a @ b
    for plan in plans(form, m, k, n):
        for dtype in (torch.float32, torch.bfloat16):
            # what lies between the rows is NaN in what is read, and stays as it is in what is written
            dA, dB, dR = R.padded(A, pad, at)[0], R.padded(Bm, pad, at)[0], R.padded(res.to(dtype), pad, at)[0]
            D, dbuf = R.padded(torch.zeros(m, n, dtype=dtype), pad, at, 7.0)
            Z, zbuf = R.padded(torch.zeros(m, n, dtype=torch.bfloat16), pad, at, 7.0)
            B.gemm_bf16_linear_run(plan, dA, dB, D, residual=dR, Z=Z)
            assert torch.equal(D.cpu(), (want + res.double()).to(dtype))
            assert torch.equal(Z.cpu(), want.to(torch.bfloat16))
            for buf, view in ((dbuf, D), (zbuf, Z)):
                assert bool((R.outside(buf, view) == 7.0).all())


def test_rows_of_other_tensors_are_not_read():
    # NaN in every row and column around the operands
    m, k, n = 33, 90, 40
    whole = R.whole
    for form in (NT, NN, TN):
        A, Bm, a, b = R.operands(form, m, k, n, whole)
        big = [torch.full((x.shape[0] + 40, x.shape[1] + 46), float("nan"), dtype=torch.bfloat16, device="cuda") for x in (A, Bm)]
        views = [y[16:16 + x.shape[0], 8:8 + x.shape[1]] for x, y in zip((A, Bm), big)]
        for x, y in zip((A, Bm), views):
            y.copy_(x)
        for plan in plans(form, m, k, n):
            D = filled(m, n, dtype=torch.float32)
            B.gemm_bf16_linear_run(plan, *views, D)
            assert torch.equal(D.cpu().double(), a @ b)


def test_accumulate_in_place():
    # a weight gradient added to what is there, several times
    n, k, rows = 130, 72, 500
    dz, x = R.whole((rows, n), 1).cuda(), R.whole((rows, k), 2).cuda()
    for plan in plans(TN, n, rows, k):
        dw = torch.ones(n, k, device="cuda")
        for _ in range(3):
            B.gemm_bf16_linear_run(plan, dz, x, dw, residual=dw)
        assert torch.equal(dw.double(), 1 + 3 * (dz.double().T @ x.double()))


def test_special_values():
    m, k, n = 20, 64, 136
    a, w = R.whole((m, k), 1), R.whole((n, k), 2)
    a[3, 5], a[7, 9] = float("nan"), float("inf")
    w[:, 5] = 1.0
    w[:, 9] = 2.0
    clean = torch.ones(m, dtype=torch.bool)
    clean[3] = clean[7] = False
    for act, code in R.ACTS.items():
        for plan in plans(NT, m, k, n):
            D = filled(m, n)
            B.gemm_bf16_linear_run(plan, a.cuda(), w.cuda(), D, activation=code)
            D = D.cpu()
            assert bool(D[3].isnan().all())
            assert bool((D[7] == float("inf")).all()), act
            v = a[clean].double() @ w.double().T
            check(D[clean], R.act(act, v), 1.2 * ACT_ERR * v.abs().clamp(min=1), torch.bfloat16)
    # RELU's gradient selects: an infinite sum behind Z <= 0 is dropped, a NaN Z is seen
    z = torch.ones(m, n, dtype=torch.bfloat16)
    z[7, :5] = -1.0
    z[0, 0] = float("nan")
    for plan in plans(NT, m, k, n):
        D = filled(m, n)
        B.gemm_bf16_linear_run(plan, a.cuda(), w.cuda(), D, activation=B.GEMM_ACT_RELU | GRAD, Z=z.cuda())
        assert bool((D[7, :5] == 0).all()) and bool((D[7, 5:] == float("inf")).all()) and bool(D[0, 0].isnan())


@pytest.mark.parametrize("act", list(R.ACTS))
def test_activations_over_their_range(act):
    # sums from the smallest to the largest magnitudes, through a product by one
    z = torch.cat([torch.linspace(-30, 30, 4001), torch.logspace(-30, 38, 500), -torch.logspace(-30, 38, 500), torch.zeros(1)])
    z = z.to(torch.bfloat16)[: 5000 // 8 * 8].reshape(-1, 8)
    one = torch.eye(8, dtype=torch.bfloat16)
    v = z.double()
    D = filled(*z.shape, dtype=torch.float32)
    plan = B.gemm_bf16_linear_plan(z.shape[0], 8, 8)
    B.gemm_bf16_linear_run(plan, z.cuda(), one.cuda(), D, activation=R.ACTS[act])
    check(D, R.act(act, v), ACT_ERR * v.abs().clamp(max=30).clamp(min=2.0 ** -100) * (R.act(act, v) != 0) + 1e-30, torch.float32)
    ones = torch.ones(z.shape, dtype=torch.bfloat16)
    dZ = filled(*z.shape)
    B.gemm_activation_backward(ones.cuda(), z.cuda(), R.ACTS[act], dZ, None)
    want = torch.where(v.abs() > 1e4, (v > 0).double(), R.slope(act, v.clamp(-1e4, 1e4))) if act != "none" else ones.double()
    check(dZ, want, torch.full_like(want, 2 * ACT_ERR), torch.bfloat16)


@pytest.mark.parametrize("act", list(R.ACTS))
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (2, 8), (65, 17), (300, 64), (1000, 130), (5000, 24), (37, 4100), (700, 777)])
def test_activation_backward(act, rows, cols):
    dy, z = R.normal((rows, cols), 1, 0.1), R.normal((rows, cols), 2, 2.0)
    slope = R.slope(act, z)
    want = dy.double() * slope
    size = dy.double().abs() * 2 * ACT_ERR
    sums, limit = want.sum(0), rows * 2.0 ** -24 * want.abs().sum(0) + size.sum(0) + 2.0 ** -100
    for pad, at in ((0, 0), (8, 8), (3, 1)):
        dY, Z = R.padded(dy, pad, at)[0], R.padded(z, pad, at)[0]
        dZ, buf = R.padded(torch.zeros_like(dy), pad, at, 7.0)
        db = filled(cols, dtype=torch.float32)
        B.gemm_activation_backward(dY, Z if act != "none" or pad else None, R.ACTS[act], dZ, db)
        check(dZ, want, size, torch.bfloat16)
        assert bool(((db.cpu().double() - sums).abs() <= limit).all())
        assert bool((R.outside(buf, dZ) == 7.0).all())
        again, only = filled(cols, dtype=torch.float32), torch.zeros_like(dZ)
        B.gemm_activation_backward(dY, Z, R.ACTS[act], None, again)    # one output alone, with the same bits
        B.gemm_activation_backward(dY, Z, R.ACTS[act], only, None)
        assert torch.equal(again, db) and torch.equal(only, dZ)
        for target in (dY, Z):                                          # in place
            y2, z2 = R.padded(dy, pad, at)[0], R.padded(z, pad, at)[0]
            out = y2 if target is dY else z2
            B.gemm_activation_backward(y2, z2, R.ACTS[act], out, again)
            assert torch.equal(out, dZ) and torch.equal(again, db)


@pytest.mark.parametrize("places", [((0, 0), (1, 0), (0, 0)), ((3, 1), (3, 1), (0, 0)), ((1, 3), (9, 11), (17, 3)), ((5, 2), (5, 3), (5, 2))])
@pytest.mark.parametrize("rows,cols", [(1, 3), (9, 5), (333, 1), (70, 249), (2100, 33), (150, 777), (440, 334)])
def test_activation_backward_of_rows_that_lie_otherwise(rows, cols, places):
    # pitches and offsets (pad, at) of dY, Z and dZ, alike modulo eight elements or not
    dy, z = R.normal((rows, cols), 1, 0.1), R.normal((rows, cols), 2, 2.0)
    want = dy.double() * R.slope("silu", z)
    size = dy.double().abs() * 2 * ACT_ERR
    dY, Z = R.padded(dy, *places[0])[0], R.padded(z, *places[1], float("nan"))[0]
    dZ, buf = R.padded(torch.zeros_like(dy), *places[2], 7.0)
    db = filled(cols, dtype=torch.float32)
    B.gemm_activation_backward(dY, Z, R.ACTS["silu"], dZ, db)
    check(dZ, want, size, torch.bfloat16)
    assert bool(((db.cpu().double() - want.sum(0)).abs() <= rows * 2.0 ** -24 * want.abs().sum(0) + size.sum(0) + 2.0 ** -100).all())
    assert bool((R.outside(buf, dZ) == 7.0).all())


def test_gradients_against_differences():
    # a layer's forward and backward calls against differences of the 64-bit layer
    m, k, n = 12, 40, 24
    x, w, b = R.normal((m, k), 1), R.normal((n, k), 2, 0.2), torch.randn(n, generator=R.gen(3))
    g = R.normal((m, n), 4)
    for act, code in R.ACTS.items():
        D, Z = filled(m, n), filled(m, n)
        B.gemm_bf16_linear_run(B.gemm_bf16_linear_plan(m, k, n), x.cuda(), w.cuda(), D, bias=b.cuda(), activation=code, Z=Z)
        dz, db = filled(m, n), filled(n, dtype=torch.float32)
        B.gemm_activation_backward(g.cuda(), Z, code, dz, db)
        dx, dw = filled(m, k, dtype=torch.float32), filled(n, k, dtype=torch.float32)
        B.gemm_bf16_linear_run(B.gemm_bf16_linear_plan(m, n, k, NN), dz, w.cuda(), dx)
        B.gemm_bf16_linear_run(B.gemm_bf16_linear_plan(n, m, k, TN), dz, x.cuda(), dw)

        def loss(x, w, b):
            return (R.act(act, x @ w.T + b) * g.double()).sum()

        args = [x.double(), w.double(), b.double()]
        for i, got in enumerate((dx, dw, db)):
            got = got.cpu().double()
            step = 1e-6
            for at in [tuple(int(v) for v in torch.randint(0, 1000, (args[i].dim(),), generator=R.gen(7 + j)) % torch.tensor(args[i].shape))
                       for j in range(12)]:
                hi, lo = [a.clone() for a in args], [a.clone() for a in args]
                hi[i][at] += step
                lo[i][at] -= step
                want = (loss(*hi) - loss(*lo)) / (2 * step)
                # dz is rounded to bfloat16 (2^-8), and so is the Z that its slope is taken of (slopes
                # change by at most 1.1 per unit): every term is off by at most 2^-6 of |g| (1 + |v|)
                v = (args[0] @ args[1].T + args[2]).abs()
                weight = g.double().abs() * (1 + v)
                other = {0: weight @ args[1].abs(), 1: weight.T @ args[0].abs(), 2: weight.sum(0)}[i]
                assert abs(got[at] - want) <= 2.0 ** -6 * other[at] + 1e-6, (act, i, at)


def test_streams_graphs_and_repeats():
    m, k, n = 200, 333, 264       # an unaligned operand: scratch from the pool in every call
    A, Bm, a, b = R.operands(NT, m, k, n, R.whole)
    bias = torch.arange(n).float()
    want = ((a @ b) + bias.double()).to(torch.bfloat16)
    dA, dB, dbias = A.cuda(), Bm.cuda(), bias.cuda()
    plan = B.gemm_bf16_linear_plan(m, k, n)
    outs = [filled(m, n) for _ in range(8)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for i, D in enumerate(outs):      # four streams at once
        B.gemm_bf16_linear_run(plan, dA, dB, D, bias=dbias, stream=streams[i % 4])
    torch.cuda.synchronize()
    for D in outs:
        assert torch.equal(D.cpu(), want)
    graphs = []
    for _ in range(2):                # two captured graphs, replayed in turn and with new inputs
        D, db, dz = filled(m, n), filled(n, dtype=torch.float32), filled(m, n)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.gemm_bf16_linear_run(plan, dA, dB, D, bias=dbias)
            B.gemm_activation_backward(D, D, B.GEMM_ACT_RELU, dz, db)
        graphs.append((graph, D, dz, db))
    dA.copy_(-A)
    want2 = ((-a @ b) + bias.double()).to(torch.bfloat16)
    for _ in range(3):
        for graph, D, dz, db in graphs:
            D.fill_(float("nan"))
            graph.replay()
    torch.cuda.synchronize()
    for graph, D, dz, db in graphs:
        assert torch.equal(D.cpu(), want2)
        relu = want2.clamp(min=0)
        assert torch.equal(dz.cpu(), relu)
        assert bool(((db.cpu().double() - relu.double().sum(0)).abs() <= m * 2.0 ** -24 * relu.double().abs().sum(0)).all())


def test_same_bits_every_time():
    m, k, n = 130, 4000, 300
    A, Bm, _, _ = R.operands(NT, m, k, n, R.normal)
    for plan in plans(NT, m, k, n):
        outs = []
        for _ in range(5):
            D = filled(m, n, dtype=torch.float32)
            B.gemm_bf16_linear_run(plan, A.cuda(), Bm.cuda(), D)
            outs.append(D)
        assert all(torch.equal(outs[0], x) for x in outs[1:])


def test_offsets_past_32_bits():
    # rows whose elements lie more than 2^31 apart: A, the residual and D
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("not enough memory")
    m, k, n = 300, 72, 136
    pitch = 2 ** 31 // 256 + 8
    a, w = R.whole((m, k), 1), R.whole((n, k), 2)
    big = torch.zeros(m, pitch, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(m, pitch, dtype=torch.bfloat16, device="cuda")
    big[:, :k] = a.cuda()
    out[:, :n] = 1.0
    B.gemm_bf16_linear_run(B.gemm_bf16_linear_plan(m, k, n), big[:, :k], w.cuda(), out[:, :n], residual=out[:, :n])
    assert torch.equal(out[:, :n].cpu(), (a.double() @ w.double().T + 1).to(torch.bfloat16))
    dz, db = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda"), filled(n, dtype=torch.float32)
    B.gemm_activation_backward(out[:, :n], out[:, :n], B.GEMM_ACT_RELU, dz, db)
    assert torch.equal(dz.cpu(), out[:, :n].cpu().clamp(min=0))


def test_trace_counts_the_launches():
    m, k, n = 64, 128, 64
    A, Bm, _, _ = R.operands(NT, m, k, n, R.whole)
    dA, dB, D = A.cuda(), Bm.cuda(), filled(m, n)
    odd = R.padded(A, 1)[0]
    plan = B.gemm_bf16_linear_plan(m, k, n)
    kind = B.GEMM_KERNEL_SKINNY if plan.path == B.GEMM_PATH_SKINNY else B.GEMM_KERNEL_TC
    B.gemm_trace_begin(16)
    B.gemm_bf16_linear_run(plan, dA, dB, D)
    B.gemm_bf16_linear_run(plan, odd, dB, D)
    torch.cuda.synchronize()
    ms, timed, counted = B.gemm_trace_collect()
    assert counted[kind] == 2 and counted[B.GEMM_KERNEL_STAGE] == 1
    assert timed[kind] == 2 and timed[B.GEMM_KERNEL_STAGE] == 1
