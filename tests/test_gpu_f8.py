"""GPU tests of the FP8 products (gemm_f8_run, gemm_f8_grouped_run) and of the
FP8 quantisation through the binding, against 64-bit references.

Two kinds of inputs.  Whole numbers with power-of-two scales: every sum is a
multiple of 2^-4 below 2^20, so fp32 results are exact whatever the order of
the additions, and are compared bit for bit.  Random values: with S the sum
of the terms' magnitudes, a block of 128 loses at most 2^-22 of its S in each
of its 132 additions (128 products and 4 partial sums; the tensor cores may
truncate instead of rounding) and the running sum 2^-24 of S per block, for
at most 128 blocks here: |error| <= (132 * 2^-22 + 128 * 2^-24) S < 2^-14 S,
plus half a unit of bfloat16 (eight significant bits: 2^-8 |D| at most)
for that output type."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import f8_ref as R

pytestmark = pytest.mark.gpu

SUM_TOL = 2.0 ** -14
BF16_TOL = 2.0 ** -8
TYPES = {R.E4M3: B.GEMM_F8_E4M3, R.E5M2: B.GEMM_F8_E5M2}


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


def on_gpu(q, pitch=None, fill=0x7F):
    """An FP8 matrix (or stack) on the GPU with the given row pitch; the bytes
    past each row are NaNs, which no result may depend on."""
    k = q.shape[-1]
    pitch = R.pad16(k) if pitch is None else pitch
    buf = torch.full(q.shape[:-1] + (pitch,), fill, dtype=torch.uint8, device="cuda")
    buf[..., :k] = q.view(torch.uint8).cuda()
    return buf.view(q.dtype)[..., :k]


def poisoned(shape, dtype, pitch, offset=0):
    """An output inside a larger buffer of a known pattern, and the buffer."""
    rows = 1
    for s in shape[:-1]:
        rows *= s
    buf = torch.full((offset + rows * pitch + 64,), -77.0, dtype=dtype, device="cuda")
    return buf[offset:offset + rows * pitch].view(*shape[:-1], pitch)[..., :shape[-1]], buf


def untouched(buf, out_count):
    return int((buf == -77.0).sum()) >= buf.numel() - out_count


def scales(m, k, n, seed, b_scale, whole, rows_b=None):
    make = R.power_scales if whole else R.any_scales
    kb, nb = (k + 127) // 128, (n + 127) // 128
    sa = make((kb, m), seed)
    sb = make((nb, kb), seed + 1) if b_scale == B.GEMM_SCALE_BLOCKS else make((kb, n), seed + 1)
    full_b = R.expand_blocks(sb, n, k) if b_scale == B.GEMM_SCALE_BLOCKS else R.expand_rows(sb, k)
    return sa, sb, R.expand_rows(sa, k), full_b


def check(got, want, S, dtype, exact):
    got = got.cpu().double()
    if exact:
        want = want.float() if dtype == torch.float32 else want.float().to(torch.bfloat16)
        assert torch.equal(got, want.double())
        return
    bound = SUM_TOL * S + (BF16_TOL * want.abs() if dtype == torch.bfloat16 else 0.0)
    bad = (got - want).abs() > bound
    assert not bool(bad.any()), "%d of %d off, first %s: %r for %r" % (
        int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())


def run_product(m, k, n, *, b_scale=B.GEMM_SCALE_BLOCKS, dtype=torch.bfloat16, whole=True, types=(R.E4M3, R.E4M3),
                seed=0, edit=None, pitch=None, offset=0, lda=None):
    make = R.whole_f8 if whole else R.normal_f8
    A, Bt = make((m, k), seed + 2, types[0]), make((n, k), seed + 3, types[1])
    sa, sb, fa, fb = scales(m, k, n, seed + 4, b_scale, whole)
    plan = B.gemm_f8_plan(m, k, n, TYPES[types[0]], TYPES[types[1]], b_scale)
    if edit:
        edit(plan)
    pitch = n if pitch is None else pitch
    D, buf = poisoned((m, n), dtype, pitch, offset)
    B.gemm_f8_run(plan, on_gpu(A, lda), sa.cuda(), on_gpu(Bt), sb.cuda(), D)
    torch.cuda.synchronize()
    want, S = R.product(A, fa, Bt, fb)
    check(D, want, S, dtype, whole)
    assert untouched(buf, m * n)
    return D


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 16, 5), (5, 130, 17), (16, 256, 300), (17, 384, 129), (33, 1000, 64),
          (64, 2048, 256), (65, 129, 127), (128, 640, 384), (129, 127, 257), (200, 1024, 1000), (256, 256, 256),
          (300, 2100, 700), (513, 520, 511), (1000, 777, 3000)]


@pytest.mark.parametrize("b_scale", [B.GEMM_SCALE_BLOCKS, B.GEMM_SCALE_ROWS])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k,n", SHAPES)
def test_product_exact(m, k, n, dtype, b_scale):
    run_product(m, k, n, dtype=dtype, b_scale=b_scale, seed=m + 7 * k)


@pytest.mark.parametrize("b_scale", [B.GEMM_SCALE_BLOCKS, B.GEMM_SCALE_ROWS])
@pytest.mark.parametrize("m,k,n", [(129, 5000, 200), (300, 8200, 300), (513, 4700, 640)])
def test_product_long_sums_with_few_tiles(m, k, n, b_scale):
    # more than 128 rows on the small tiles, with the sum split over CTAs: as planned, and with 128 rows a tile
    plan = B.gemm_f8_plan(m, k, n, b_scale=b_scale)
    assert plan.path == B.GEMM_PATH_SKINNY and plan.split_k > 1
    for edit in (None, _set(path=B.GEMM_PATH_SKINNY, bm=128, bn=128, split_k=8)):
        run_product(m, k, n, b_scale=b_scale, dtype=torch.float32, seed=13, edit=edit)
        run_product(m, k, n, b_scale=b_scale, dtype=torch.bfloat16, seed=14, pitch=n + 3, offset=1, edit=edit)
        run_product(m, k, n, b_scale=b_scale, dtype=torch.bfloat16, whole=False, seed=15, edit=edit)


@pytest.mark.parametrize("types", [(R.E4M3, R.E5M2), (R.E5M2, R.E4M3), (R.E5M2, R.E5M2)])
@pytest.mark.parametrize("m,k,n", [(3, 500, 200), (300, 700, 400)])
def test_product_types(m, k, n, types):
    run_product(m, k, n, types=types, dtype=torch.float32, seed=5)


@pytest.mark.parametrize("b_scale", [B.GEMM_SCALE_BLOCKS, B.GEMM_SCALE_ROWS])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k,n", [(1, 8192, 512), (40, 3000, 700), (100, 4096, 1024), (700, 2500, 900), (1024, 4096, 512)])
def test_product_random(m, k, n, dtype, b_scale):
    run_product(m, k, n, dtype=dtype, b_scale=b_scale, whole=False, seed=11)


def _set(**kw):
    def edit(plan):
        for name, v in kw.items():
            setattr(plan, name, v)
    return edit


SKINNY = [dict(path=B.GEMM_PATH_SKINNY, bm=bm, bn=128, split_k=s) for bm in (16, 32, 64, 128) for s in (1, 2, 4, 8)]
TENSOR = [dict(path=B.GEMM_PATH_TENSOR, bm=256, bn=bn, split_k=1) for bn in (128, 256)]


@pytest.mark.parametrize("b_scale", [B.GEMM_SCALE_BLOCKS, B.GEMM_SCALE_ROWS])
@pytest.mark.parametrize("cfg", SKINNY + TENSOR, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_product_every_configuration(cfg, b_scale):
    # more rows than a skinny tile, a ragged n, fewer K blocks than the largest split, and more
    for m, k, n in [(150, 700, 300), (20, 2500, 129)]:
        run_product(m, k, n, b_scale=b_scale, edit=_set(**cfg), dtype=torch.float32, seed=21)
        run_product(m, k, n, b_scale=b_scale, edit=_set(**cfg), dtype=torch.bfloat16, seed=22, pitch=n + 3, offset=1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pitch,offset", [(300, 0), (304, 8), (301, 0), (303, 1), (512, 3)])
def test_product_output_pitch_and_alignment(dtype, pitch, offset):
    for m in (9, 280):
        run_product(m, 400, 300, dtype=dtype, pitch=pitch, offset=offset, lda=464, seed=31)


def test_product_nan_and_inf_stay_in_their_row():
    m, k, n = 300, 512, 260
    A, Bt = R.whole_f8((m, k), 1), R.whole_f8((n, k), 2)
    raw = A.view(torch.uint8)
    raw[7, 300] = 0x7F                      # the e4m3 NaN
    sa, sb, fa, fb = scales(m, k, n, 3, B.GEMM_SCALE_BLOCKS, True)
    sa[1, 130] = float("inf")
    fa = R.expand_rows(sa, k)
    for rows in (m, 131):
        D, _ = poisoned((rows, n), torch.float32, n)
        B.gemm_f8_run(B.gemm_f8_plan(rows, k, n), on_gpu(A[:rows]), sa[:, :rows].contiguous().cuda(), on_gpu(Bt),
                      sb.cuda(), D)
        D = D.cpu()
        assert bool(D[7].isnan().all()) and not bool(D[130].isfinite().any())
        keep = [i for i in range(rows) if i not in (7, 130)]
        want = R.product(raw[keep].view(R.E4M3), fa[keep], Bt, fb)[0]
        assert torch.equal(D[keep].double(), want)


def test_product_same_bits_twice_and_on_another_stream():
    m, k, n = 48, 4096, 640
    A, Bt = R.normal_f8((m, k), 1), R.normal_f8((n, k), 2)
    sa, sb, _, _ = scales(m, k, n, 3, B.GEMM_SCALE_BLOCKS, False)
    args = [on_gpu(A), sa.cuda(), on_gpu(Bt), sb.cuda()]
    plan = B.gemm_f8_plan(m, k, n)
    first = torch.empty(m, n, device="cuda")
    B.gemm_f8_run(plan, *args, first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = [torch.empty(m, n, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for D in again:
        B.gemm_f8_run(plan, *args, D, stream=side)
    side.synchronize()
    assert all(torch.equal(first, D) for D in again)


def test_product_in_a_cuda_graph():
    m, k, n = 8, 1024, 512
    A, Bt = R.whole_f8((m, k), 1), R.whole_f8((n, k), 2)
    sa, sb, fa, fb = scales(m, k, n, 3, B.GEMM_SCALE_BLOCKS, True)
    args = [on_gpu(A), sa.cuda(), on_gpu(Bt), sb.cuda()]
    plan = B.gemm_f8_plan(m, k, n)
    D = torch.empty(m, n, device="cuda")
    B.gemm_f8_run(plan, *args, D)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gemm_f8_run(plan, *args, D)
    D.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(D.cpu().double(), R.product(A, fa, Bt, fb)[0])


# -------------------------------------------------------------- by expert --

SIZES = {"even": [64, 64, 64, 64], "ragged": [1, 0, 130, 257, 3, 0, 0, 64], "one": [77], "none": [0, 0, 0],
         "first": [300, 0, 0], "last": [0, 0, 300], "ones": [1] * 40, "many": [3, 0, 5, 1] * 75, "big": [513, 255, 256]}


def grouped_inputs(sizes, k, n, m, seed, b_scale, first=0):
    g = len(sizes)
    kb, nb = (k + 127) // 128, (n + 127) // 128
    A, Bt = R.whole_f8((m, k), seed), R.whole_f8((g, n, k), seed + 1)
    sa = R.power_scales((kb, m), seed + 2)
    sb = R.power_scales((g, nb, kb) if b_scale == B.GEMM_SCALE_BLOCKS else (kb, g * n), seed + 3)
    off = [first]
    for s in sizes:
        off.append(off[-1] + s)
    want = torch.full((m, n), float("nan"), dtype=torch.float64)
    for i in range(g):
        lo, hi = off[i], off[i + 1]
        fb = R.expand_blocks(sb[i], n, k) if b_scale == B.GEMM_SCALE_BLOCKS else R.expand_rows(
            sb[:, i * n:(i + 1) * n], k)
        want[lo:hi] = R.product(A[lo:hi], R.expand_rows(sa[:, lo:hi], k), Bt[i], fb)[0]
    return A, sa, Bt, sb, off, want


def run_grouped_rows(sizes, k, n, *, extra=0, first=0, seed=0, b_scale=B.GEMM_SCALE_BLOCKS, dtype=torch.float32,
                     edit=None):
    m = max(1, first + sum(sizes) + extra)
    A, sa, Bt, sb, off, want = grouped_inputs(sizes, k, n, m, seed, b_scale, first)
    plan = B.gemm_f8_grouped_plan(B.GEMM_GROUP_ROWS, len(sizes), m, k, n, b_scale=b_scale)
    if edit:
        edit(plan)
    D, buf = poisoned((m, n), dtype, n + 5)
    B.gemm_f8_grouped_run(plan, on_gpu(A), sa.cuda(), on_gpu(Bt), sb.cuda(),
                          torch.tensor(off, dtype=torch.int32, device="cuda"), D)
    torch.cuda.synchronize()
    D = D.cpu()
    lo, hi = off[0], off[-1]
    assert torch.equal(D[lo:hi].double(), want[lo:hi].to(dtype).double())
    assert bool((D[:lo] == -77).all()) and bool((D[hi:] == -77).all()), "rows outside every group were written"
    assert untouched(buf, m * n)


@pytest.mark.parametrize("b_scale", [B.GEMM_SCALE_BLOCKS, B.GEMM_SCALE_ROWS])
@pytest.mark.parametrize("k,n", [(256, 128), (300, 200), (1100, 513)])
@pytest.mark.parametrize("name", list(SIZES))
def test_grouped_rows(name, k, n, b_scale):
    run_grouped_rows(SIZES[name], k, n, b_scale=b_scale, seed=41)


@pytest.mark.parametrize("cfg", SKINNY + TENSOR, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_grouped_rows_every_configuration(cfg):
    run_grouped_rows([5, 0, 140, 33, 1, 260], 520, 200, edit=_set(**cfg), seed=51)


@pytest.mark.parametrize("sizes", [[300, 0, 200], [500, 1, 0], [0, 0, 450]])
def test_grouped_rows_long_sums_with_few_tiles(sizes):
    # the plan knows the mean of the groups only: one may hold every row
    plan = B.gemm_f8_grouped_plan(B.GEMM_GROUP_ROWS, 3, sum(sizes), 4700, 300)
    assert plan.path == B.GEMM_PATH_SKINNY and plan.split_k > 1
    run_grouped_rows(sizes, 4700, 300, seed=52)
    run_grouped_rows(sizes, 4700, 300, seed=52, edit=_set(path=B.GEMM_PATH_SKINNY, bm=128, bn=128, split_k=8))


def test_grouped_rows_spare_capacity_and_first_offset():
    run_grouped_rows([3, 0, 20], 256, 160, extra=50, first=4, seed=61)
    run_grouped_rows([300, 10, 270], 256, 160, extra=500, first=9, seed=62, dtype=torch.bfloat16)


def test_grouped_rows_neighbours_do_not_leak():
    # a group whose rows are NaN next to others: their results stay exact
    sizes, k, n = [20, 13, 200], 384, 150
    A, sa, Bt, sb, off, want = grouped_inputs(sizes, k, n, sum(sizes), 71, B.GEMM_SCALE_BLOCKS)
    A.view(torch.uint8)[20:33] = 0x7F
    D = torch.empty(sum(sizes), n, device="cuda")
    B.gemm_f8_grouped_run(B.gemm_f8_grouped_plan(B.GEMM_GROUP_ROWS, 3, sum(sizes), k, n), on_gpu(A), sa.cuda(), on_gpu(Bt),
                          sb.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"), D)
    D = D.cpu().double()
    assert bool(D[20:33].isnan().all())
    assert torch.equal(D[:20], want[:20]) and torch.equal(D[33:], want[33:])


@pytest.mark.parametrize("bad", [[0, 10, 5, 60], [-5, 20, 40, 60], [0, 20, 1000, 2000], [50, 40, 30, 20],
                                 [2 ** 31 - 1] * 4, [-2 ** 31] * 4])
def test_grouped_offsets_are_clamped(bad):
    # offsets outside the matrix or out of order are clamped by the kernels:
    # no access leaves the operands, and D stays inside its buffer
    m, k, n = 60, 256, 140
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    A, sa, Bt, sb, _, _ = grouped_inputs([20, 20, 20], k, n, m, 81, B.GEMM_SCALE_BLOCKS)
    D, buf = poisoned((m, n), torch.float32, n)
    B.gemm_f8_grouped_run(B.gemm_f8_grouped_plan(B.GEMM_GROUP_ROWS, 3, m, k, n), on_gpu(A), sa.cuda(), on_gpu(Bt), sb.cuda(),
                          off, D)
    X = torch.randn(m, 70, device="cuda")
    kp = B.gemm_f8_padded_k(m, 3)
    Q, S = torch.zeros(70, kp, dtype=R.E4M3, device="cuda"), torch.zeros(kp // 128, 70, device="cuda")
    B.gemm_f8_quantize_cols(X, Q, S, off)
    W = torch.empty(3, 70, 70, device="cuda")
    B.gemm_f8_grouped_run(B.gemm_f8_grouped_plan(B.GEMM_GROUP_K, 3, 70, kp, 70, b_scale=B.GEMM_SCALE_ROWS), Q, S, Q, S,
                          off, W)
    torch.cuda.synchronize()
    assert untouched(buf, m * n)


def run_grouped_k(sizes, n1, n2, *, seed=0, dtype=torch.float32, b_scale=B.GEMM_SCALE_ROWS, edit=None):
    g, rows = len(sizes), max(1, sum(sizes))
    kp = R.padded_k(rows, g)
    assert kp == B.gemm_f8_padded_k(rows, g)
    at = R.padded_starts(sizes)
    A, Bt = R.whole_f8((n1, kp), seed), R.whole_f8((n2, kp), seed + 1)
    for i, s in enumerate(sizes):   # the padding of each group is zero, what lies behind the last is NaN
        A[:, at[i] + s:at[i + 1]] = 0
        Bt[:, at[i] + s:at[i + 1]] = 0
    A.view(torch.uint8)[:, at[-1]:] = 0x7F
    Bt.view(torch.uint8)[:, at[-1]:] = 0x7F
    kb = kp // 128
    sa = R.power_scales((kb, n1), seed + 2)
    sb = R.power_scales((kb, n2) if b_scale == B.GEMM_SCALE_ROWS else ((n2 + 127) // 128, kb), seed + 3)
    fb = R.expand_rows(sb, kp) if b_scale == B.GEMM_SCALE_ROWS else R.expand_blocks(sb, n2, kp)
    fa = R.expand_rows(sa, kp)
    plan = B.gemm_f8_grouped_plan(B.GEMM_GROUP_K, g, n1, kp, n2, b_scale=b_scale)
    if edit:
        edit(plan)
    D, buf = poisoned((g, n1, n2), dtype, n2 + 2)
    off = [0]
    for s in sizes:
        off.append(off[-1] + s)
    B.gemm_f8_grouped_run(plan, on_gpu(A), sa.cuda(), on_gpu(Bt), sb.cuda(),
                          torch.tensor(off, dtype=torch.int32, device="cuda"), D)
    torch.cuda.synchronize()
    for i in range(g):
        c = slice(at[i], at[i + 1])
        want = R.product(A[:, c], fa[:, c], Bt[:, c], fb[:, c])[0]
        assert torch.equal(D[i].cpu().double(), want.to(dtype).double()), "group %d" % i
    assert untouched(buf, g * n1 * n2)


@pytest.mark.parametrize("n1,n2", [(128, 256), (200, 130), (513, 300), (7, 5)])
@pytest.mark.parametrize("name", list(SIZES))
def test_grouped_k(name, n1, n2):
    run_grouped_k(SIZES[name], n1, n2, seed=91)


def test_grouped_k_long_sums_with_few_tiles():
    kp = B.gemm_f8_padded_k(9000, 2)
    plan = B.gemm_f8_grouped_plan(B.GEMM_GROUP_K, 2, 200, kp, 130, b_scale=B.GEMM_SCALE_ROWS)
    assert plan.path == B.GEMM_PATH_SKINNY and plan.split_k > 1
    run_grouped_k([8000, 1000], 200, 130, seed=95)
    run_grouped_k([0, 9000], 200, 130, seed=96)


def test_grouped_k_block_scales_and_bf16():
    run_grouped_k([130, 0, 40], 260, 200, b_scale=B.GEMM_SCALE_BLOCKS, seed=92)
    run_grouped_k([130, 0, 40], 260, 200, dtype=torch.bfloat16, seed=93)


@pytest.mark.parametrize("cfg", SKINNY + TENSOR, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_grouped_k_every_configuration(cfg):
    run_grouped_k([130, 0, 400, 1, 128], 140, 200, edit=_set(**cfg), seed=94)


# ------------------------------------------------------------ quantisation --

def values(rows, cols, seed, dtype):
    x = torch.randn(rows, cols, generator=R.gen(seed)) * torch.exp(3 * torch.randn(1, cols, generator=R.gen(seed + 1)))
    if rows > 2 and cols > 2:
        x[rows // 2] = 0
        x[0, 0] = 0
    return x.to(dtype)


def pitched(x, pad):
    buf = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device="cuda")
    buf[:, :x.shape[1]] = x.cuda()
    return buf[:, :x.shape[1]]


def same_f8(got, want):
    return torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


QSHAPES = [(1, 1), (1, 128), (3, 777), (128, 128), (130, 260), (257, 1000), (64, 4096)]


@pytest.mark.parametrize("f8", [R.E4M3, R.E5M2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", QSHAPES)
def test_quantise_rows_and_blocks(rows, cols, dtype, f8):
    x = values(rows, cols, 100 + rows, dtype)
    kb, rb = (cols + 127) // 128, (rows + 127) // 128
    for pad in (0, 3, 16):
        X = pitched(x, pad)
        for mode, ref, shape in ((B.GEMM_SCALE_ROWS, R.quantise_rows, (kb, rows)),
                                 (B.GEMM_SCALE_BLOCKS, R.quantise_blocks, (rb, kb))):
            Q = on_gpu(torch.zeros(rows, cols).to(f8), R.pad16(cols) + pad)
            S = torch.full(shape, -1.0, device="cuda")
            B.gemm_f8_quantize(X, Q, S, mode)
            q, s = ref(x, f8)
            assert torch.equal(S.cpu(), s) and same_f8(Q.contiguous(), q)


@pytest.mark.parametrize("f8", [R.E4M3, R.E5M2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", QSHAPES)
def test_quantise_cols(rows, cols, dtype, f8):
    x = values(rows, cols, 200 + rows, dtype)
    kp = R.padded_k(rows, 1)
    for pad in (0, 5):
        Q = torch.full((cols, kp + 16), 0x55, dtype=torch.uint8, device="cuda")
        S = torch.full((kp // 128, cols), -1.0, device="cuda")
        B.gemm_f8_quantize_cols(pitched(x, pad), Q.view(f8)[:, :kp], S)
        xt = torch.zeros(cols, kp)
        xt[:, :rows] = x.float().T
        q, s = R.quantise_rows(xt, f8)
        assert torch.equal(S.cpu(), s) and same_f8(Q[:, :kp].contiguous(), q)
        assert bool((Q[:, kp:] == 0x55).all())


@pytest.mark.parametrize("name", list(SIZES))
def test_quantise_cols_by_group(name):
    sizes, cols = SIZES[name], 150
    rows = max(1, sum(sizes))
    x = values(rows, cols, 300, torch.bfloat16)
    g, kp, at = len(sizes), R.padded_k(rows, len(sizes)), R.padded_starts(sizes)
    Q = torch.full((cols, kp), 0x55, dtype=torch.uint8, device="cuda")
    S = torch.full((kp // 128, cols), -1.0, device="cuda")
    off = [0]
    for s in sizes:
        off.append(off[-1] + s)
    B.gemm_f8_quantize_cols(x.cuda(), Q.view(R.E4M3), S, torch.tensor(off, dtype=torch.int32, device="cuda"))
    Q, S = Q.cpu(), S.cpu()
    for i in range(g):
        xt = torch.zeros(cols, at[i + 1] - at[i])
        xt[:, :sizes[i]] = x[off[i]:off[i + 1]].float().T
        q, s = R.quantise_rows(xt, R.E4M3)
        assert torch.equal(S[at[i] // 128:at[i + 1] // 128], s)
        assert torch.equal(Q[:, at[i]:at[i + 1]], q.view(torch.uint8))
    assert bool((Q[:, at[-1]:] == 0x55).all()) and bool((S[at[-1] // 128:] == -1).all())


def test_quantise_special_values():
    x = torch.randn(130, 256, generator=R.gen(7))
    x[3, 5], x[9, 200], x[50] = float("inf"), float("nan"), 0.0
    x[60, :128] = 1e-42                       # below the smallest normal number
    x[70, :128] = 3.0e38
    X = x.cuda()
    Q, S = on_gpu(torch.zeros(130, 256).to(R.E4M3)), torch.empty(2, 130, device="cuda")
    B.gemm_f8_quantize(X, Q, S)
    Q, S = Q.cpu().contiguous().view(torch.uint8), S.cpu()
    assert S[0, 3].item() == float("inf") and Q[3, 5].item() & 0x7F == 0x7F
    assert bool((Q[3, :5] & 0x7F == 0).all()) and bool((Q[3, 6:128] & 0x7F == 0).all())
    assert Q[9, 200].item() & 0x7F == 0x7F and bool(S[1, 9].isfinite())
    others = [c for c in range(128, 256) if c != 200]
    y = x.clone()
    y[9, 200], y[3, 5] = 0.0, 0.0
    q, s = R.quantise_rows(y, R.E4M3)
    assert torch.equal(Q[9, others], q.view(torch.uint8)[9, others]) and S[1, 9] == s[1, 9]
    assert S[0, 50].item() == R.SCALE_MIN and bool((Q[50] == 0).all())
    assert S[0, 60].item() == R.SCALE_MIN and S[0, 70].item() == s[0, 70].item()
    assert bool((Q[70, :128] == 0x7E).all())   # 448


def test_linear_backward_chain():
    """dX and dW of D = X W^T through the quantisers and products together,
    against the products of the quantised values in 64 bits."""
    m, k, n = 300, 260, 200
    x, dy = values(m, k, 1, torch.bfloat16), (torch.randn(m, n, generator=R.gen(2)) * 0.02).to(torch.bfloat16)
    w = torch.randn(n, k, generator=R.gen(3)) * 0.02
    wt, ws = R.quantise_blocks(w.T.contiguous(), R.E4M3)          # (k, n)
    dq, ds = on_gpu(torch.zeros(m, n).to(R.E4M3)), torch.empty((n + 127) // 128, m, device="cuda")
    B.gemm_f8_quantize(dy.cuda(), dq, ds)
    dx = torch.empty(m, k, device="cuda")
    B.gemm_f8_run(B.gemm_f8_plan(m, n, k), dq, ds, on_gpu(wt), ws.cuda(), dx)
    q, s = R.quantise_rows(dy, R.E4M3)
    want, S = R.product(q, R.expand_rows(s, n), wt, R.expand_blocks(ws, k, n))
    check(dx, want, S, torch.float32, False)
    kp = B.gemm_f8_padded_k(m)
    parts = []
    for t in (dy, x):
        Q, sc = torch.empty(t.shape[1], kp, dtype=R.E4M3, device="cuda"), torch.empty(kp // 128, t.shape[1], device="cuda")
        B.gemm_f8_quantize_cols(t.cuda(), Q, sc)
        parts += [Q, sc]
    dw = torch.empty(n, k, device="cuda")
    B.gemm_f8_run(B.gemm_f8_plan(n, kp, k, b_scale=B.GEMM_SCALE_ROWS), *parts, dw)
    refs = []
    for t in (dy, x):
        tt = torch.zeros(t.shape[1], kp)
        tt[:, :m] = t.float().T
        q, s = R.quantise_rows(tt, R.E4M3)
        refs += [q, R.expand_rows(s, kp)]
    want, S = R.product(*refs)
    check(dw, want, S, torch.float32, False)
