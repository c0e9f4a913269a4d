"""GPU tests of the balance loss and its gradient with so many rows that the
kernels go round their loops many times, the running sums are flushed, and the
grids reach their limits.

Tolerances.  p of a row and lse: q as in test_gpu_balance.py.  Means over the
rows: a lane adds up at most rows / 2048 rows (the fewest rows at once: 256 CTAs
of eight warps), and joins at most 300 sums, one after the other.  With logits of which one is 0 and the others
-infinity, p is 1 or 0 and every sum a whole number below 2^24, thus exact."""

import math

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import layer_ref as R
from tests.test_gpu_balance import COEF, forward

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# rows, experts, slots per row: 32 and more rows per lane on 152 SMs, with 1 to 32 lanes to a row
CASES = [(4000000, 4, 1), (4000001, 8, 1), (3200000, 16, 2), (1700000, 33, 2), (260000, 256, 8), (130000, 512, 4), (100000, 1024, 2),
         (90001, 601, 40)]


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


def routes(rows, e, k, g):
    """Slots with dropped ones, and padding at the end and in the middle."""
    index = torch.randint(0, e, (rows, k), generator=g, device="cuda", dtype=torch.int32)
    index[torch.rand(rows, k, generator=g, device="cuda") < 0.05] = -1
    index[rows // 2:rows // 2 + rows // 9] = -1
    index[rows - rows // 8:] = e
    return index


def padded(x, pad):
    buf = torch.full((x.shape[0], x.shape[1] + pad), 7.0, dtype=x.dtype, device="cuda")
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]], buf


@pytest.mark.parametrize("dtype,pad", [(F32, 0), (BF16, 0), (BF16, 1), (F32, 4)])
@pytest.mark.parametrize("rows,e,k", CASES)
def test_many_rows(rows, e, k, dtype, pad):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + e)
    index = routes(rows, e, k, g)
    taken = (index >= 0) & (index < e)
    used = taken.any(1)
    counts = torch.bincount(index[taken].long(), minlength=e)
    t = int(used.sum())
    f = counts.double() / counts.sum()

    # one logit of 0, the others -infinity
    only = torch.randint(0, e, (rows,), generator=g, device="cuda")
    x = torch.full((rows, e), -math.inf, dtype=dtype, device="cuda")
    x[torch.arange(rows, device="cuda"), only] = 0.0
    x[~used] = float("nan")                              # padding is not read
    X = padded(x, pad)[0]
    o = forward(X, index)
    assert torch.equal(o["counts"].long(), counts) and int(o["used"]) == t
    assert torch.equal(o["offsets"].long(), torch.nn.functional.pad(counts.cumsum(0), (1, 0)))
    assert torch.equal(o["lse"], torch.where(used, 0.0, math.inf))
    sums = torch.bincount(only[used], minlength=e)
    assert torch.equal(o["probs"], sums.float() / torch.tensor(float(t), device="cuda"))
    want = COEF * e * (f * sums.double() / t).sum().item()
    assert abs(o["loss"].item() - want) <= (e / 32 + 12) * 2.0 ** -24 * want
    del x, X

    # any logits, both passes
    x = (torch.randn(rows, e, generator=g, device="cuda") * 2).to(dtype)
    X = padded(x, pad)[0]
    o = forward(X, index)
    xd = x.double()
    lse = torch.where(used, torch.logsumexp(xd, 1), math.inf)
    p = torch.where(used[:, None], torch.softmax(xd, 1), 0.0)
    del xd
    most = x.float().abs().max().item()
    q = (2 * most + 8) * 2.0 ** -23 + (e / 32 + 8) * 2.0 ** -24
    assert torch.equal(o["lse"][~used], lse[~used].float())
    assert bool(((o["lse"].double() - lse)[used].abs() <= q + 2.0 ** -23 * lse[used].abs()).all())
    mean = q + (rows / 2048 + 300) * 2.0 ** -24
    probs = p.sum(0) / t
    assert bool(((o["probs"].double() - probs).abs() <= mean * probs).all())
    want = COEF * e * (f * probs).sum().item()
    assert abs(o["loss"].item() - want) <= (mean + (e / 32 + 12) * 2.0 ** -24) * want

    dr = (torch.randn(rows, e, generator=g, device="cuda") * (COEF / t)).to(dtype)
    dR = padded(dr, pad)[0]
    dX, buf = padded(torch.zeros_like(dr), pad)
    B.gemm_balance_backward(X, o["lse"], o["counts"], o["used"], COEF, torch.full((1,), 1.5, device="cuda"), dR, dX)
    mix = (p * f).sum(1, keepdim=True)
    scale = 1.5 * COEF * e / t
    want, size = scale * p * (f - mix) + dr.double(), scale * p * (f + mix) + dr.double().abs()
    size *= 2 * q + (e / 32 + 12) * 2.0 ** -24 + lse.where(used, torch.zeros_like(lse)).abs()[:, None] * 2.0 ** -23
    assert bool(((dX.double() - want).abs() <= size + R.HALF_STEP[dtype] * (want.abs() + size) + 1e-38).all())
    assert torch.equal(dX[~used], dr[~used])
    assert bool((buf[:, e:] == 7.0).all())
