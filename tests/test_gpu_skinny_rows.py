"""GPU tests of int8 products of few rows whose k is not a multiple of 16 (the
CUDA-core kernel for rows that start at any byte), bit for bit against int64
sums, through the plain, the requantising and the allocation-free entry point;
and how their time compares with the tensor cores' at the next multiple of 16."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_int8_matrix_gb300 import build
    build.build()
    B.load()


def operands(m, k, n, seed):
    g = torch.Generator().manual_seed(seed)
    A = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8)
    Bt = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8)
    return A, Bt


def product(A, Bt):
    """int64 sums: every partial sum of the fp64 product is a whole number below 2^53."""
    return A.double() @ Bt.double().T


def run(call, A, Bt):
    """C inside a larger buffer whose ends stay as they were."""
    m, n = A.shape[0], Bt.shape[0]
    buf = torch.full((m * n + 128,), -7, dtype=torch.int32, device="cuda")
    C = buf[64:64 + m * n].view(m, n)
    plan = B.gemm_i8_plan(m, A.shape[1], n)
    assert plan.path == B.GEMM_PATH_SKINNY
    call(plan, A.cuda(), Bt.cuda(), C)
    torch.cuda.synchronize()
    assert bool((buf[:64] == -7).all()) and bool((buf[64 + m * n:] == -7).all())
    return C.cpu()


@pytest.mark.parametrize("k", [1, 2, 3, 15, 17, 31, 33, 255, 257, 271, 273, 1001, 4094, 8191])
def test_exact(k):
    for m, n in [(1, 1), (1, 300), (2, 33), (7, 31), (8, 32), (9, 97), (16, 5), (17, 64), (31, 300), (33, 1), (63, 40), (64, 129)]:
        A, Bt = operands(m, k, n, 1000 * m + k + n)
        want = product(A, Bt)
        assert torch.equal(run(B.gemm_i8_run, A, Bt).double(), want), (m, n)
        assert torch.equal(run(B.gemm_i8_run_noalloc, A, Bt).double(), want), (m, n)


def test_exact_at_the_limits():
    # the longest k, every product of the largest magnitude and of one sign: the
    # sum is the largest that int32 holds for this k
    for m, n, k in [(2, 5, 131071), (40, 3, 131069)]:
        A = torch.full((m, k), -128, dtype=torch.int8)
        Bt = torch.full((n, k), -128, dtype=torch.int8)
        Bt[1] = 127
        want = product(A, Bt)
        assert torch.equal(run(B.gemm_i8_run, A, Bt).double(), want)


@pytest.mark.parametrize("m,k,n", [(1, 777, 300), (5, 4095, 64), (40, 333, 257), (64, 1001, 96)])
def test_requantised(m, k, n):
    A, Bt = operands(m, k, n, m + k)
    g = torch.Generator().manual_seed(n)
    rs, cs = torch.rand(m, generator=g) / 100 + 1e-3, torch.rand(n, generator=g) / 100 + 1e-3
    D = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    B.gemm_i8_run_requant(B.gemm_i8_plan(m, k, n), A.cuda(), Bt.cuda(), rs.cuda(), cs.cuda(), D)
    want = (product(A, Bt).float() * rs[:, None]) * cs
    assert torch.equal(D.cpu(), want.to(torch.bfloat16))


def test_rows_of_neighbours_do_not_leak():
    # the words around a row hold its neighbours' bytes: other rows' values change nothing in this one's results
    m, k, n = 20, 301, 70
    A, Bt = operands(m, k, n, 5)
    first = run(B.gemm_i8_run, A, Bt)
    A2, Bt2 = A.clone(), Bt.clone()
    A2[::2] = 127
    Bt2[1::2] = -128
    again = run(B.gemm_i8_run, A2, Bt2)
    assert torch.equal(again[1::2, ::2], first[1::2, ::2])
    assert torch.equal(again.double(), product(A2, Bt2))


def median_us(call, reps=15):
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    times = []
    for i in range(reps + 3):
        flush.zero_()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        if i >= 3:
            times.append(a.elapsed_time(b) * 1e3)
    return sorted(times)[len(times) // 2]


@pytest.mark.parametrize("m,k,n", [(64, 4095, 256), (55, 1940, 620), (16, 4095, 4096), (64, 1001, 1001)])
def test_time_beside_the_next_multiple_of_16(m, k, n):
    # dp4a on CUDA cores has about a thirtieth of the tensor cores' rate, but
    # products of so few rows are not bound by it: 16 times is allowed.  A byte
    # load per multiply-add takes 50 to 180 times.
    def us(kk):
        A, Bt = operands(m, kk, n, 1)
        A, Bt, C = A.cuda(), Bt.cuda(), torch.empty(m, n, dtype=torch.int32, device="cuda")
        plan = B.gemm_i8_plan(m, kk, n)
        return median_us(lambda: B.gemm_i8_run(plan, A, Bt, C))

    here, even = us(k), us((k + 15) // 16 * 16)
    assert here <= 16 * even, "%.1f us against %.1f" % (here, even)
