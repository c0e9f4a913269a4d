"""GPU tests of the layer norm, the balance loss and their gradients on matrices
whose elements lie more than 2^31 apart: the same bits as with a small pitch that
takes the same kernels."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B

pytestmark = pytest.mark.gpu

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


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip("not enough memory")


def matrix(x, pitch):
    """x as the first columns of rows of `pitch` elements."""
    view = torch.empty(x.shape[0], pitch, dtype=x.dtype, device="cuda")[:, :x.shape[1]]
    view.copy_(x)
    return view


# few rows, the ring, and rows that are not aligned; (40 rows: a CTA each, two passes backward)
@pytest.mark.parametrize("rows,d,far,near,dtype", [(700, 1032, 2 ** 22, 1040, BF16), (700, 1032, 2 ** 22 + 1, 1033, BF16),
                                                   (40, 1032, 2 ** 26, 1040, BF16), (1300, 250, 2 ** 21 + 1, 251, F32),
                                                   (1300, 120, 2 ** 21, 128, F32)])
def test_layer_norm(rows, d, far, near, dtype):
    room(80)
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    x, r, dy = (torch.randn(rows, d, generator=g, device="cuda").to(dtype) for _ in range(3))
    w, b = torch.randn(d, generator=g, device="cuda"), torch.randn(d, generator=g, device="cuda")
    outs = []
    for pitch in (near, far):
        X, Rr, Y = matrix(x, pitch), matrix(r, pitch), matrix(dy, pitch)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        B.gemm_layer_norm(X, Rr, w, b, 1e-5, X, mean, rstd, Y)         # h in place of x
        h, y = X.contiguous(), Y.contiguous()
        dW, dB = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        Y.copy_(dy)
        B.gemm_layer_norm_backward(Y, X, w, mean, rstd, Rr, Rr, dW, dB)   # dx in place of dr
        outs.append((h, y, mean, rstd, Rr.contiguous(), dW, dB))
        del X, Rr, Y
    assert torch.equal(outs[0][0], (x.float() + r.float()).to(dtype))
    for a, c in zip(*outs):
        assert torch.equal(a, c)


@pytest.mark.parametrize("rows,e,far,near,dtype", [(2200, 64, 2 ** 20, 68, F32), (2200, 33, 2 ** 20 + 1, 34, BF16), (40, 300, 2 ** 26, 304, BF16)])
def test_balance(rows, e, far, near, dtype):
    room(40)
    g = torch.Generator(device="cuda")
    g.manual_seed(e)
    x, dr = (torch.randn(rows, e, generator=g, device="cuda").to(dtype) for _ in range(2))
    index = torch.randint(-1, e, (rows, 2), generator=g, device="cuda", dtype=torch.int32)
    outs = []
    for pitch in (near, far):
        X, dX = matrix(x, pitch), matrix(dr, pitch)
        counts, offsets, used = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (e, e + 1, 1))
        lse, probs, loss = (torch.empty(n, device="cuda") for n in (rows, e, 1))
        B.gemm_balance(X, index, 0.1, counts, offsets, used, lse, probs, loss)
        B.gemm_balance_backward(X, lse, counts, used, 0.1, loss, dX, dX)
        outs.append((counts, offsets, used, lse, probs, loss, dX.contiguous()))
        del X, dX
    assert bool(outs[0][5].isfinite().all())
    for a, c in zip(*outs):
        assert torch.equal(a, c)
