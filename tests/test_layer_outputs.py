"""Host-side test: the bfloat16 layer's entry points refuse an output that is an
operand or another output, except where a declaration allows it in place.  Every
other pointer of a call is its own, so that each refusal has one cause, and the
refusal comes before any CUDA call."""

import ctypes
import itertools

import pytest

from dense_int8_matrix_gb300 import binding as B
from dense_int8_matrix_gb300 import build as build_mod

P = 4096   # addresses that are never read: every call here is refused


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def linear(lib, act, out, A, B_, bias, Z, residual, D):
    plan = B.gemm_bf16_linear_plan_for_sms(24, 24, 24, 152)
    return lib.gemm_bf16_linear_run(ctypes.byref(plan), A, 24, B_, 24, bias, act, Z, 24, residual, 24, out, D, 24, None)


# call, operands, outputs, pairs that may be the same
CASES = {
    "linear": (lambda lib, **p: linear(lib, B.GEMM_ACT_SILU, B.GEMM_OUT_F32, **p), ["A", "B_", "bias", "residual"], ["Z", "D"],
               {("D", "residual")}),
    "linear bf16": (lambda lib, **p: linear(lib, B.GEMM_ACT_NONE, B.GEMM_OUT_BF16, **p), ["A", "B_", "bias", "residual"], ["Z", "D"],
                    {("D", "residual")}),
    "linear gradient": (lambda lib, **p: linear(lib, B.GEMM_ACT_GELU | B.GEMM_ACT_GRADIENT, B.GEMM_OUT_BF16, **p),
                        ["A", "B_", "bias", "residual", "Z"], ["D"], {("D", "residual")}),
    "activation": (lambda lib, dY, Z, dZ, dbias: lib.gemm_activation_backward(dY, 24, Z, 24, B.GEMM_ACT_GELU, 16, 24, dZ, 24, dbias, None),
                   ["dY", "Z"], ["dZ", "dbias"], {("dZ", "dY"), ("dZ", "Z")}),
    "layer norm": (lambda lib, X, R, W, bias, H, mean, rstd, Y: lib.gemm_layer_norm(
        X, 24, R, 24, W, bias, 1e-5, 2, 2, 16, 24, H, 24, mean, rstd, Y, 24, None),
        ["X", "R", "W", "bias"], ["H", "mean", "rstd", "Y"], {("H", "X"), ("H", "R")}),
    "layer norm backward": (lambda lib, dY, H, W, mean, rstd, dR, dX, dW, dbias: lib.gemm_layer_norm_backward(
        dY, 24, H, 24, W, mean, rstd, dR, 24, 2, 2, 16, 24, dX, 24, dW, dbias, None),
        ["dY", "H", "W", "mean", "rstd", "dR"], ["dX", "dW", "dbias"], {("dX", "dY"), ("dX", "dR")}),
    "balance": (lambda lib, X, index, counts, offsets, used, lse, probs, loss: lib.gemm_balance(
        X, 8, 2, 16, 8, index, 2, 1.0, counts, offsets, used, lse, probs, loss, None),
        ["X", "index"], ["counts", "offsets", "used", "lse", "probs", "loss"], set()),
    "balance backward": (lambda lib, X, lse, counts, used, dloss, dR, dX: lib.gemm_balance_backward(
        X, 8, 2, 16, 8, lse, counts, used, 1.0, dloss, dR, 8, dX, 8, None),
        ["X", "lse", "counts", "used", "dloss", "dR"], ["dX"], {("dX", "dR")}),
}
PAIRS = [(name, a, b) for name, (_, ins, outs, allowed) in CASES.items()
         for a, b in itertools.chain(itertools.product(outs, ins), itertools.combinations(outs, 2)) if (a, b) not in allowed]


@pytest.mark.parametrize("name,a,b", PAIRS)
def test_an_output_that_is_an_operand_or_another_output(lib, name, a, b):
    call, ins, outs, _ = CASES[name]
    p = {n: P * (i + 1) for i, n in enumerate(ins + outs)}
    p[a] = p[b]
    assert call(lib, **p) == B.GEMM_ERR_INVALID_ARG
