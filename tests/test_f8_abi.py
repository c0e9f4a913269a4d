"""Host-side checks of the 8-bit operators' entry points: plans, and argument
errors that come back before any CUDA call."""

import ctypes

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from dense_int8_matrix_gb300 import build as build_mod

INV, MIS = B.GEMM_ERR_INVALID_ARG, B.GEMM_ERR_MISALIGNED
P = 4096          # an aligned address that is never read: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def test_plan_struct_and_fields(lib):
    p = B.gemm_f8_plan_for_sms(B.GEMM_GROUP_NONE, 1, 1000, 777, 3000, 152)
    assert ctypes.sizeof(B.gemm_plan_f8) == 104
    assert (p.version, p.m, p.k, p.n, p.groups) == (B.GEMM_PLAN_F8_VERSION, 1000, 777, 3000, 1)
    assert (p.a_type, p.b_type, p.b_scale) == (B.GEMM_F8_E4M3, B.GEMM_F8_E4M3, B.GEMM_SCALE_BLOCKS)
    for m in (1, 16, 17, 100, 500, 5000):
        for sms in (1, 132, 152):
            for mode, groups in ((B.GEMM_GROUP_NONE, 1), (B.GEMM_GROUP_ROWS, 8), (B.GEMM_GROUP_K, 8)):
                q = B.gemm_f8_plan_for_sms(mode, groups, m, 4096, 2048, sms)
                assert q.path in (B.GEMM_PATH_TENSOR, B.GEMM_PATH_SKINNY)
                if q.path == B.GEMM_PATH_TENSOR:
                    assert q.bm == 256 and q.bn in (128, 256) and q.split_k == 1
                else:
                    assert q.bm in (16, 32, 64, 128) and q.bn == 128 and q.split_k in (1, 2, 4, 8)


def test_plan_takes_the_tiles_that_fill_the_sms(lib):
    def plan(m, k, n, mode=B.GEMM_GROUP_NONE, groups=1):
        return B.gemm_f8_plan_for_sms(mode, groups, m, k, n, 152)

    assert plan(300, 16384, 640).path == B.GEMM_PATH_SKINNY and plan(300, 16384, 640).split_k == 8
    assert plan(2000, 2000, 2000).path == B.GEMM_PATH_TENSOR       # enough large tiles
    assert plan(300, 16384, 9000).path == B.GEMM_PATH_TENSOR
    assert plan(600, 600, 600).path == B.GEMM_PATH_TENSOR          # a sum too short to split
    assert plan(1000, 4096, 512, B.GEMM_GROUP_ROWS, 3).split_k > 1
    big = 2 ** 30                                                  # nothing overflows at the limits
    assert plan(big, big, big).path == B.GEMM_PATH_TENSOR
    assert plan(big, 128, 1000, B.GEMM_GROUP_ROWS, 1024).path == B.GEMM_PATH_TENSOR


def test_plan_refusals(lib):
    def plan(mode=0, groups=1, m=5, k=128, n=5, a=0, b=0, s=1, sms=152, out=True):
        p = B.gemm_plan_f8()
        return lib.gemm_f8_plan_for_sms(mode, groups, m, k, n, a, b, s, sms, ctypes.byref(p) if out else None)

    assert plan() == B.GEMM_OK
    for bad in (dict(m=0), dict(k=0), dict(n=-1), dict(m=2 ** 31), dict(a=2), dict(b=-1), dict(s=2), dict(mode=3),
                dict(mode=-1), dict(groups=2), dict(groups=0), dict(sms=0), dict(out=False),
                dict(mode=1, groups=1025), dict(mode=1, groups=0), dict(mode=1, groups=1024, n=2 ** 22),
                dict(mode=2, groups=4, k=130), dict(mode=2, groups=1024, m=2 ** 22)):
        assert plan(**bad) == INV, bad
    p = B.gemm_plan_f8()
    assert lib.gemm_f8_grouped_plan(0, 1, 5, 128, 5, 0, 0, 1, ctypes.byref(p)) == INV
    assert lib.gemm_f8_plan(0, 128, 5, 0, 0, 1, ctypes.byref(p)) == INV
    assert lib.gemm_f8_plan(5, 128, 5, 0, 0, 1, None) == INV


def test_run_refusals(lib):
    p = B.gemm_f8_plan_for_sms(B.GEMM_GROUP_NONE, 1, 64, 200, 100, 152)

    def run(plan=p, A=P, lda=208, sa=P, Bt=P, ldb=208, sb=P, out=B.GEMM_OUT_BF16, D=P, ldd=100):
        return lib.gemm_f8_run(ctypes.byref(plan) if plan else None, A, lda, sa, Bt, ldb, sb, out, D, ldd, None)

    for bad in (dict(plan=None), dict(A=None), dict(Bt=None), dict(sa=None), dict(sb=None), dict(D=None),
                dict(lda=192), dict(ldb=199), dict(ldd=99), dict(out=2), dict(out=0), dict(lda=2 ** 40)):
        assert run(**bad) == INV, bad
    for bad in (dict(A=P + 8), dict(Bt=P + 1), dict(lda=200), dict(ldb=216), dict(sa=P + 2), dict(sb=P + 1),
                dict(D=P + 1), dict(out=B.GEMM_OUT_F32, D=P + 2)):
        assert run(**bad) == MIS, bad
    for field, value in (("version", 9), ("m", 0), ("k", -1), ("a_type", 5), ("group_mode", 1), ("groups", 2),
                         ("path", 7), ("bm", 48), ("bn", 96), ("split_k", 3)):
        q = B.gemm_f8_plan_for_sms(B.GEMM_GROUP_NONE, 1, 64, 200, 100, 152)
        setattr(q, field, value)
        assert run(plan=q) == INV, field
    g = B.gemm_f8_plan_for_sms(B.GEMM_GROUP_ROWS, 4, 64, 200, 100, 152)
    assert run(plan=g) == INV                                             # grouped plans need offsets
    gr = lib.gemm_f8_grouped_run
    assert gr(ctypes.byref(g), P, 208, P, P, 208, P, None, 1, P, 100, None) == INV
    assert gr(ctypes.byref(p), P, 208, P, P, 208, P, P, 1, P, 100, None) == INV
    assert gr(ctypes.byref(g), P, 208, P, P, 208, P, P + 2, 1, P, 100, None) == MIS


def test_quantise_refusals(lib):
    def rows(X=P, t=1, r=5, c=300, ldx=300, f=0, mode=0, Q=P, ldq=304, s=P):
        return lib.gemm_f8_quantize(X, t, r, c, ldx, f, mode, Q, ldq, s, None)

    for bad in (dict(X=None), dict(Q=None), dict(s=None), dict(t=0), dict(t=3), dict(r=0), dict(c=0), dict(ldx=299),
                dict(ldq=299), dict(f=2), dict(mode=2), dict(r=2 ** 31)):
        assert rows(**bad) == INV, bad
    assert rows(X=P + 1) == MIS and rows(t=2, X=P + 2) == MIS and rows(s=P + 2) == MIS

    def cols(X=P, t=1, r=300, c=20, ldx=20, f=0, off=None, g=1, Q=P, ldq=384, s=P):
        return lib.gemm_f8_quantize_cols(X, t, r, c, ldx, f, off, g, Q, ldq, s, None)

    for bad in (dict(X=None), dict(Q=None), dict(s=None), dict(g=0), dict(g=2), dict(off=P, g=1025), dict(ldq=256),
                dict(off=P, g=9, ldq=1279), dict(f=3), dict(r=0)):
        assert cols(**bad) == INV, bad
    assert cols(Q=P + 8) == MIS and cols(ldq=392) == MIS and cols(off=P + 1) == MIS


def test_padded_k(lib):
    assert [B.gemm_f8_padded_k(r) for r in (1, 128, 129, 4096)] == [128, 128, 256, 4096]
    assert B.gemm_f8_padded_k(300, 9) == 1408 and B.gemm_f8_padded_k(1, 1) == 128
    assert B.gemm_f8_padded_k(0) == 0 and B.gemm_f8_padded_k(5, 0) == 0
    for rows, groups in ((40, 40), (900, 300), (1, 3)):   # as many groups as possible with one row too many
        worst = sum((s + 127) // 128 * 128 for s in [1] * (min(rows, groups) - 1) + [rows - min(rows, groups) + 1])
        assert worst <= B.gemm_f8_padded_k(rows, groups)


def test_norm_refusals(lib):
    for name in ("gemm_norm_f8", "gemm_norm_i8"):
        f = getattr(lib, name)

        def run(X=P, ldx=64, R=P, ldr=64, W=P, eps=1e-6, t=1, rows=4, d=64, H=P * 2, ldh=64, rstd=P, Q=P, ldq=64, s=P):
            return f(X, ldx, R, ldr, W, eps, t, rows, d, H, ldh, rstd, Q, ldq, s, None)

        for bad in (dict(X=None), dict(W=None), dict(Q=None), dict(s=None), dict(H=None), dict(t=0), dict(rows=0),
                    dict(d=0), dict(d=B.GEMM_NORM_MAX_D + 1, ldx=40000, ldr=40000, ldh=40000, ldq=40000), dict(eps=-1.0),
                    dict(eps=float("nan")), dict(ldx=63), dict(ldr=60), dict(ldh=1), dict(ldq=63),
                    dict(H=P, ldh=72)):
            assert run(**bad) == INV, bad
        for bad in (dict(X=P + 1), dict(R=P + 1), dict(W=P + 2), dict(rstd=P + 1), dict(s=P + 2), dict(t=2, X=P + 2)):
            assert run(**bad) == MIS, bad

    def back(dY=P, ly=64, H=P, lh=64, W=P, rstd=P, dR=None, lr=0, t=1, rows=4, d=64, dX=P, lx=64, dW=P):
        return lib.gemm_norm_backward(dY, ly, H, lh, W, rstd, dR, lr, t, rows, d, dX, lx, dW, None)

    for bad in (dict(dY=None), dict(H=None), dict(W=None), dict(rstd=None), dict(dX=None), dict(t=5), dict(rows=-1),
                dict(d=0), dict(ly=63), dict(lx=63), dict(lh=63), dict(dR=P, lr=63), dict(dR=P, lr=72)):
        assert back(**bad) == INV, bad
    for bad in (dict(dY=P + 1), dict(dX=P + 1), dict(rstd=P + 1), dict(dW=P + 2), dict(dR=P + 1, lr=64)):
        assert back(**bad) == MIS, bad


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour")
def test_no_device_means_error(lib):
    p = B.gemm_f8_plan_for_sms(B.GEMM_GROUP_NONE, 1, 64, 128, 100, 152)
    assert lib.gemm_f8_run(ctypes.byref(p), P, 128, P, P, 128, P, 1, P, 100, None) == B.GEMM_ERR_CUDA
    assert lib.gemm_norm_backward(P, 64, P, 64, P, P, None, 0, 1, 4, 64, P, 64, P, None) == B.GEMM_ERR_CUDA
    assert lib.gemm_f8_quantize(P, 1, 5, 300, 300, 0, 0, P, 304, P, None) == B.GEMM_ERR_CUDA


def test_binding_checks_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        B.gemm_f8_quantize(x, torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(1, 4))   # host tensors
    with pytest.raises(TypeError):
        B.gemm_f8_grouped_run(B.gemm_plan_f8(), x, x, x, x, None, x)
