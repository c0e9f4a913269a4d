"""Host-side checks of the bfloat16 layer's entry points: plans, argument errors
that come back before any CUDA call, and the binding's checks of tensors."""

import ctypes

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from dense_int8_matrix_gb300 import build as build_mod
from tests.test_binding_device import BF16, F32, I32, calls, on  # noqa: F401  (a fixture)

INV, MIS = B.GEMM_ERR_INVALID_ARG, B.GEMM_ERR_MISALIGNED
P = 4096          # an aligned address that is never read: every call here is refused first
FORMS = (B.GEMM_FORM_NT, B.GEMM_FORM_NN, B.GEMM_FORM_TN)
BIG = 2 ** 30


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def test_plan_struct_and_fields(lib):
    assert ctypes.sizeof(B.gemm_plan_linear) == 88
    p = B.gemm_bf16_linear_plan_for_sms(1000, 777, 3000, 152, B.GEMM_FORM_NN)
    assert (p.version, p.form, p.m, p.k, p.n, p.num_sms) == (B.GEMM_PLAN_LINEAR_VERSION, B.GEMM_FORM_NN, 1000, 777, 3000, 152)
    for form in FORMS:
        for m in (1, 16, 17, 64, 100, 500, 5000, BIG):
            for k, n in ((1, 1), (777, 3000), (8192, 8192), (BIG, BIG), (4096, 128)):
                for sms in (1, 132, 152):
                    q = B.gemm_bf16_linear_plan_for_sms(m, k, n, sms, form)
                    if q.path == B.GEMM_PATH_TENSOR:
                        assert q.bm == 256 and q.bn in (128, 256) and q.split_k == 1
                    else:
                        assert q.path == B.GEMM_PATH_SKINNY and q.bn == 128 and q.split_k in (1, 2, 4, 8)
                        assert q.bm in ((64, 128) if form == B.GEMM_FORM_TN else (16, 32, 64, 128))


def test_plan_refusals(lib):
    def plan(form=0, m=5, k=128, n=5, sms=152, out=True):
        p = B.gemm_plan_linear()
        return lib.gemm_bf16_linear_plan_for_sms(form, m, k, n, sms, ctypes.byref(p) if out else None)

    assert plan() == B.GEMM_OK
    for bad in (dict(m=0), dict(k=0), dict(n=-1), dict(m=BIG + 1), dict(k=2 ** 31), dict(form=3), dict(form=-1), dict(sms=0),
                dict(out=False)):
        assert plan(**bad) == INV, bad
    assert lib.gemm_bf16_linear_plan(0, 5, 128, 5, None) == INV
    p = B.gemm_plan_linear()
    assert lib.gemm_bf16_linear_plan(0, 0, 128, 5, ctypes.byref(p)) == INV


def test_linear_run_refusals(lib):
    def run(plan=None, A=P, lda=128, Bm=P, ldb=128, bias=0, act=0, Z=0, ldz=0, R=0, ldr=0, out=B.GEMM_OUT_BF16, D=P, ldd=24, **edit):
        p = plan or B.gemm_bf16_linear_plan_for_sms(16, 128, 24, 152, edit.pop("form", 0))
        for k, v in edit.items():
            setattr(p, k, v)
        return lib.gemm_bf16_linear_run(ctypes.byref(p), A, lda, Bm, ldb, bias, act, Z, ldz, R, ldr, out, D, ldd, None)

    for bad in (dict(A=0), dict(Bm=0), dict(D=0), dict(lda=127), dict(ldb=100), dict(ldd=23), dict(out=2), dict(out=0), dict(act=5),
                dict(act=-1), dict(act=32), dict(act=B.GEMM_ACT_GRADIENT | B.GEMM_ACT_GELU), dict(act=B.GEMM_ACT_GRADIENT | 7),
                dict(Z=P, ldz=23), dict(R=P, ldr=23), dict(R=P, ldr=32), dict(version=2), dict(path=7), dict(bm=48), dict(bn=64),
                dict(split_k=3), dict(m=0), dict(k=2 ** 31), dict(lda=2 ** 31 + 8),
                dict(form=B.GEMM_FORM_NN, ldb=23), dict(form=B.GEMM_FORM_TN, lda=15, ldb=24)):
        assert run(**bad) == INV, bad
    for bad in (dict(A=P + 1), dict(Bm=P + 1), dict(D=P + 1), dict(out=B.GEMM_OUT_F32, D=P + 2), dict(bias=P + 2),
                dict(Z=P + 1, ldz=24), dict(R=P + 1, ldr=24), dict(out=B.GEMM_OUT_F32, R=P + 2, ldr=24)):
        assert run(**bad) == MIS, bad
    assert lib.gemm_bf16_linear_run(None, P, 128, P, 128, 0, 0, 0, 0, 0, 0, 1, P, 24, None) == INV


def test_activation_backward_refusals(lib):
    def run(dY=P, lddy=24, Z=2 * P, ldz=24, act=B.GEMM_ACT_GELU, rows=16, cols=24, dZ=3 * P, lddz=24, db=P):
        return lib.gemm_activation_backward(dY, lddy, Z, ldz, act, rows, cols, dZ, lddz, db, None)

    for bad in (dict(dY=0), dict(Z=0), dict(dZ=0, db=0), dict(act=5), dict(act=17), dict(rows=0), dict(cols=BIG + 1), dict(lddy=23),
                dict(ldz=23), dict(lddz=23), dict(dZ=P, lddz=32), dict(dZ=2 * P, lddz=32)):
        assert run(**bad) == INV, bad
    for bad in (dict(dY=P + 1), dict(Z=P + 1), dict(dZ=P + 1), dict(db=P + 2)):
        assert run(**bad) == MIS, bad


def test_layer_norm_refusals(lib):
    def run(X=P, ldx=24, R=2 * P, ldr=24, W=P, bias=P, eps=1e-5, xt=1, yt=1, rows=16, d=24, H=3 * P, ldh=24, mean=P, rstd=P, Y=4 * P, ldy=24):
        return lib.gemm_layer_norm(X, ldx, R, ldr, W, bias, eps, xt, yt, rows, d, H, ldh, mean, rstd, Y, ldy, None)

    for bad in (dict(X=0), dict(W=0), dict(Y=0), dict(H=0), dict(xt=0), dict(yt=3), dict(rows=0), dict(d=0), dict(ldx=23), dict(ldr=23),
                dict(ldh=23), dict(ldy=23), dict(eps=-1.0), dict(eps=float("nan")), dict(H=P, ldh=32), dict(H=2 * P, ldh=32),
                dict(d=B.GEMM_NORM_MAX_D + 1, ldx=2 ** 20, ldr=2 ** 20, ldh=2 ** 20, ldy=2 ** 20)):
        assert run(**bad) == INV, bad
    for bad in (dict(X=P + 1), dict(xt=2, X=P + 2), dict(yt=2, Y=P + 2), dict(R=P + 1), dict(H=P + 1), dict(Y=P + 1), dict(W=P + 2),
                dict(bias=P + 2), dict(mean=P + 1), dict(rstd=P + 1)):
        assert run(**bad) == MIS, bad


def test_layer_norm_backward_refusals(lib):
    def run(dY=P, lddy=24, H=2 * P, ldh=24, W=P, mean=P, rstd=P, dR=3 * P, lddr=24, xt=1, yt=1, rows=16, d=24, dX=4 * P, lddx=24, dW=P, db=P):
        return lib.gemm_layer_norm_backward(dY, lddy, H, ldh, W, mean, rstd, dR, lddr, xt, yt, rows, d, dX, lddx, dW, db, None)

    for bad in (dict(dY=0), dict(H=0), dict(W=0), dict(mean=0), dict(rstd=0), dict(dX=0), dict(xt=3), dict(yt=0), dict(rows=BIG + 1),
                dict(d=0), dict(lddy=23), dict(ldh=23), dict(lddr=23), dict(lddx=23), dict(dX=3 * P, lddx=32), dict(dX=P, lddx=32),
                dict(dX=P, yt=2), dict(d=B.GEMM_NORM_MAX_D + 1, lddy=2 ** 20, ldh=2 ** 20, lddr=2 ** 20, lddx=2 ** 20)):
        assert run(**bad) == INV, bad
    for bad in (dict(dY=P + 1), dict(H=P + 1), dict(W=P + 2), dict(mean=P + 2), dict(rstd=P + 2), dict(dR=P + 1), dict(dX=P + 1),
                dict(dW=P + 1), dict(db=P + 1), dict(xt=2, H=P + 2), dict(yt=2, dY=P + 2)):
        assert run(**bad) == MIS, bad


def test_balance_refusals(lib):
    def run(X=P, ldx=8, xt=2, rows=16, e=8, index=P, k=2, coef=1.0, counts=P, offsets=P, used=P, lse=P, probs=P, loss=P):
        return lib.gemm_balance(X, ldx, xt, rows, e, index, k, coef, counts, offsets, used, lse, probs, loss, None)

    for bad in (dict(X=0), dict(index=0), dict(counts=0), dict(used=0), dict(lse=0), dict(probs=0), dict(loss=0), dict(xt=0), dict(ldx=7),
                dict(rows=0), dict(e=0), dict(e=1025, ldx=2000), dict(k=0), dict(rows=BIG, k=2)):
        assert run(**bad) == INV, bad
    for bad in (dict(X=P + 2), dict(index=P + 1), dict(counts=P + 1), dict(offsets=P + 2), dict(used=P + 1), dict(lse=P + 1),
                dict(probs=P + 1), dict(loss=P + 2), dict(xt=1, X=P + 1)):
        assert run(**bad) == MIS, bad


def test_balance_backward_refusals(lib):
    def run(X=P, ldx=8, xt=2, rows=16, e=8, lse=P, counts=P, used=P, coef=1.0, dloss=P, dR=2 * P, lddr=8, dX=3 * P, lddx=8):
        return lib.gemm_balance_backward(X, ldx, xt, rows, e, lse, counts, used, coef, dloss, dR, lddr, dX, lddx, None)

    for bad in (dict(X=0), dict(lse=0), dict(counts=0), dict(used=0), dict(dloss=0), dict(dX=0), dict(xt=3), dict(ldx=7), dict(lddr=7),
                dict(lddx=7), dict(rows=0), dict(e=0), dict(e=1025, ldx=2000, lddr=2000, lddx=2000), dict(dX=2 * P, lddx=9)):
        assert run(**bad) == INV, bad
    for bad in (dict(X=P + 2), dict(lse=P + 2), dict(counts=P + 1), dict(used=P + 1), dict(dloss=P + 1), dict(dR=P + 2), dict(dX=P + 2)):
        assert run(**bad) == MIS, bad


def test_outputs_that_are_operands_are_refused(lib):
    p = B.gemm_bf16_linear_plan_for_sms(16, 24, 24, 152)
    A, Bm, Z, R, D = (P * i for i in range(1, 6))
    for a, b, z, r, d in ((D, Bm, Z, R, D), (A, D, Z, R, D), (A, Bm, D, R, D), (A, Bm, A, R, D), (A, Bm, Bm, R, D), (A, Bm, R, R, D)):
        assert lib.gemm_bf16_linear_run(ctypes.byref(p), a, 24, b, 24, 0, B.GEMM_ACT_SILU, z, 24, r, 24, B.GEMM_OUT_BF16, d, 24, None) == INV
    act = B.GEMM_ACT_SILU | B.GEMM_ACT_GRADIENT
    assert lib.gemm_bf16_linear_run(ctypes.byref(p), A, 24, Bm, 24, 0, act, D, 24, R, 24, B.GEMM_OUT_BF16, D, 24, None) == INV
    X, R, H, Y, W, dW = (P * i for i in range(1, 7))
    for y, mean, rstd in ((X, 0, 0), (R, 0, 0), (H, 0, 0), (Y, dW, dW)):
        assert lib.gemm_layer_norm(X, 24, R, 24, W, 0, 1e-5, 1, 1, 16, 24, H, 24, mean, rstd, y, 24, None) == INV
    for dx, dw in ((H, dW), (Y, W)):
        assert lib.gemm_layer_norm_backward(X, 24, H, 24, W, P, P, R, 24, 1, 1, 16, 24, dx, 24, dw, W, None) == INV
    assert lib.gemm_balance_backward(X, 8, 2, 16, 8, P, P, P, 1.0, P, R, 8, X, 8, None) == INV


# ------------------------------------------------------------ the binding --

def linear_plan(form):
    p = B.gemm_plan_linear()
    p.m, p.k, p.n, p.form = 16, 64, 24, form
    return p


CALLS = {
    "gemm_bf16_linear_run": (
        lambda a, b, d, bias, z, r: B.gemm_bf16_linear_run(linear_plan(0), a, b, d, bias, B.GEMM_ACT_SILU, z, r),
        [((16, 64), BF16), ((24, 64), BF16), ((16, 24), BF16), ((24,), F32), ((16, 24), BF16), ((16, 24), BF16)]),
    "gemm_bf16_linear_run nn": (
        lambda a, b, d: B.gemm_bf16_linear_run(linear_plan(1), a, b, d), [((16, 64), BF16), ((64, 24), BF16), ((16, 24), F32)]),
    "gemm_bf16_linear_run tn": (
        lambda a, b, d: B.gemm_bf16_linear_run(linear_plan(2), a, b, d), [((64, 16), BF16), ((64, 24), BF16), ((16, 24), F32)]),
    "gemm_activation_backward": (
        lambda dy, z, dz, db: B.gemm_activation_backward(dy, z, B.GEMM_ACT_GELU, dz, db),
        [((16, 24), BF16), ((16, 24), BF16), ((16, 24), BF16), ((24,), F32)]),
    "gemm_layer_norm": (
        lambda x, r, w, b, h, mean, rstd, y: B.gemm_layer_norm(x, r, w, b, 1e-5, h, mean, rstd, y),
        [((5, 24), F32), ((5, 24), F32), ((24,), F32), ((24,), F32), ((5, 24), F32), ((5,), F32), ((5,), F32), ((5, 24), BF16)]),
    "gemm_layer_norm_backward": (
        lambda dy, h, w, mean, rstd, dr, dx, dw, db: B.gemm_layer_norm_backward(dy, h, w, mean, rstd, dr, dx, dw, db),
        [((5, 24), BF16), ((5, 24), F32), ((24,), F32), ((5,), F32), ((5,), F32), ((5, 24), F32), ((5, 24), F32), ((24,), F32), ((24,), F32)]),
    "gemm_balance": (
        lambda x, i, c, o, u, lse, p, loss: B.gemm_balance(x, i, 0.1, c, o, u, lse, p, loss),
        [((5, 8), F32), ((5, 2), I32), ((8,), I32), ((9,), I32), ((1,), I32), ((5,), F32), ((8,), F32), ((1,), F32)]),
    "gemm_balance_backward": (
        lambda x, lse, c, u, dl, dr, dx: B.gemm_balance_backward(x, lse, c, u, 0.1, dl, dr, dx),
        [((5, 8), BF16), ((5,), F32), ((8,), I32), ((1,), I32), ((1,), F32), ((5, 8), BF16), ((5, 8), BF16)]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_only_fitting_tensors_of_the_current_device_reach_the_library(name, calls):  # noqa: F811
    call, wanted = CALLS[name]

    def tensors(devs):
        return [on(d, *shape, dtype=dtype) for d, (shape, dtype) in zip(devs, wanted)]

    n = len(wanted)
    call(*tensors([0] * n))
    assert calls == [name.split()[0]]
    with pytest.raises(ValueError, match="current device"):
        call(*tensors([1] * n))
    for i in range(n):
        for dev in (1, -1):
            devs = [0] * n
            devs[i] = dev
            with pytest.raises(ValueError, match="device"):
                call(*tensors(devs))
        good = tensors([0] * n)
        shape, dtype = wanted[i]
        more = on(0, shape[0] + 1, *shape[1:], dtype=dtype)             # another shape
        with pytest.raises((ValueError, TypeError)):
            call(*good[:i], more, *good[i + 1:])
        other = on(0, *shape, dtype=torch.float64)                      # another type
        with pytest.raises(TypeError):
            call(*good[:i], other, *good[i + 1:])
        if len(shape) == 2:
            turned = on(0, *shape[::-1], dtype=dtype).T                  # rows that are not contiguous
            turned.device_index = 0
            with pytest.raises(ValueError):
                call(*good[:i], turned, *good[i + 1:])
    assert calls == [name.split()[0]], "a refused call reached the library"
