"""GPU tests of the activations' left tails, relative to their value there: a form
that cancels (1 + erf, 1 - sigmoid) loses every digit and would pass an absolute
limit.  fp32 outputs of a product by one.

Limits, in units of 2^-23 of the value.  exp(-x) within 2 + 1.16 x of itself, and
the rounding of x = v^2 / 2 adds x / 2.  GELU: the polynomial's fit 2.3; its
argument's rounding 1.5, at most 2.7 times as much in erfc(x) exp(x^2), 4; its eight steps 3; three
products 1.5; exp 2 + 0.83 v^2: 12.8 + 0.83 v^2.  Sigmoid: exp 2 + 1.16 |u|, sum and
reciprocal 1.5, product 0.5: 4 + 1.16 |u|, where the u of GELU_TANH is off by
seven roundings, 3.5 |u|, besides.  Slopes: the same for each term, and half a
unit for each product and sum.  Where exp or 1 / (1 + exp) passes below 2^-126 it
is zero: at most 128 * 2^-126 = 2^-119 is lost."""

import math

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

U, LOST = 2.0 ** -23, 2.0 ** -119
TWICE, CUBE = 2 * math.sqrt(2 / math.pi), 0.044715


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


def values():
    v = torch.cat([torch.linspace(-110, 0, 8000), torch.linspace(-15, 15, 16000), -torch.logspace(-30, 4, 400), torch.logspace(-30, 4, 400)])
    return v.to(torch.bfloat16)[: v.numel() // 8 * 8].reshape(-1, 8)


def plans(m, k, n):
    yield B.gemm_bf16_linear_plan(m, k, n)
    p = B.gemm_bf16_linear_plan(m, k, n)
    p.path, p.bm, p.bn, p.split_k = B.GEMM_PATH_TENSOR, 256, 256, 1
    yield p


def sigmoid_parts(name, v):
    u = v if name == "silu" else TWICE * (v + CUBE * v ** 3)
    return u, torch.sigmoid(u), (1.16 if name == "silu" else 4.66) * u.abs() + 4


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_value(name):
    z = values()
    v = z.double()
    want = R.act(name, v)
    units = 12.8 + 0.83 * v ** 2 if name == "gelu" else sigmoid_parts(name, v)[2]
    for plan in plans(z.shape[0], 8, 8):
        D = torch.full(z.shape, float("nan"), device="cuda")
        B.gemm_bf16_linear_run(plan, z.cuda(), torch.eye(8, dtype=torch.bfloat16, device="cuda"), D, activation=R.ACTS[name])
        err = (D.cpu().double() - want).abs()
        assert bool((err <= units * U * want.abs() + LOST).all()), (err / (units * U * want.abs() + LOST)).max()


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_slope(name):
    z = values()
    v = z.double()
    if name == "gelu":
        phi, tail = torch.exp(-v ** 2 / 2) / math.sqrt(2 * math.pi), torch.special.erfc(-v / math.sqrt(2)) / 2
        want = tail + v * phi
        limit = (12.8 + 0.83 * v ** 2) * tail.clamp(max=1) + (3.5 + 0.83 * v ** 2) * v.abs() * phi + 0.5 * want.abs()
        limit = torch.where(v > 0, limit + 0.5, limit)                    # 1 - tail
    else:
        u, s, units = sigmoid_parts(name, v)
        du = torch.ones_like(v) if name == "silu" else TWICE * (1 + 3 * CUBE * v ** 2)
        t = 1 - s
        want = s + v * s * t * du
        # both terms by the error of s and of 1 - s, five roundings in the second, the sum
        limit = units * s + v.abs() * du * s * (t * (units + 5) + s * units + 0.5) + 0.5 * want.abs()
    for plan in plans(z.shape[0], 8, 8):
        one = torch.zeros(z.shape, dtype=torch.bfloat16, device="cuda")
        one[:, 0] = 1.0
        D = torch.full(z.shape, float("nan"), device="cuda")
        w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
        w[:, 0] = 1.0
        B.gemm_bf16_linear_run(plan, one, w, D, activation=R.ACTS[name] | B.GEMM_ACT_GRADIENT, Z=z.cuda())
        err = (D.cpu().double() - want).abs()
        assert bool((err <= limit * U + LOST * (1 + v.abs()) * 8).all()), (err / (limit * U + LOST)).max()
