"""The bfloat16 layer's kernels against a producer that lets them start early: each
operand in turn, and each output's old content, is written about 50 us after the
kernels behind have been allowed to start (tests/cuda/late_writer.cu).  A kernel
that reads an operand, or writes an output, before the work in front of it has
ended gives other outputs."""

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B
from tests.test_gpu_pdl import writer  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def linear(m, k, n, form=B.GEMM_FORM_NT, act=B.GEMM_ACT_GELU, out=BF16, pad=0, **edit):
    a = (k, m) if form == B.GEMM_FORM_TN else (m, k)
    b = (n, k) if form == B.GEMM_FORM_NT else (k, n)
    plan = B.gemm_bf16_linear_plan(m, k, n, form)
    for name, value in edit.items():
        setattr(plan, name, value)
    grad = bool(act & B.GEMM_ACT_GRADIENT)
    ins = dict(A=(a, BF16), B=(b, BF16), bias=((n,), F32), R=((m, n), out))
    outs = dict(D=((m, n), out))
    (ins if grad else outs)["Z"] = ((m, n), BF16)
    return ins, outs, pad, lambda t: B.gemm_bf16_linear_run(plan, t["A"], t["B"], t["D"], t["bias"], act, t["Z"], t["R"])


def activation(rows, cols, pads=0):
    return (dict(dY=((rows, cols), BF16), Z=((rows, cols), BF16)), dict(dZ=((rows, cols), BF16), db=((cols,), F32)), pads,
            lambda t: B.gemm_activation_backward(t["dY"], t["Z"], B.GEMM_ACT_SILU, t["dZ"], t["db"]))


def norm(rows, d, tx=BF16, pad=0):
    m = (rows, d)
    return (dict(X=(m, tx), R=(m, tx), W=((d,), F32), bias=((d,), F32)),
            dict(H=(m, tx), mean=((rows,), F32), rstd=((rows,), F32), Y=(m, BF16)), pad,
            lambda t: B.gemm_layer_norm(t["X"], t["R"], t["W"], t["bias"], 1e-5, t["H"], t["mean"], t["rstd"], t["Y"]))


def norm_backward(rows, d, tx=BF16, pad=0):
    m = (rows, d)
    return (dict(dY=(m, BF16), H=(m, tx), W=((d,), F32), mean=((rows,), F32), rstd=((rows,), F32), dR=(m, tx)),
            dict(dX=(m, tx), dW=((d,), F32), db=((d,), F32)), pad,
            lambda t: B.gemm_layer_norm_backward(t["dY"], t["H"], t["W"], t["mean"], t["rstd"], t["dR"], t["dX"], t["dW"], t["db"]))


def balance(rows, e, k=2, tx=F32, pad=0):
    return (dict(X=((rows, e), tx), index=((rows, k), I32)),
            dict(counts=((e,), I32), offsets=((e + 1,), I32), used=((1,), I32), lse=((rows,), F32), probs=((e,), F32), loss=((1,), F32)), pad,
            lambda t: B.gemm_balance(t["X"], t["index"], 0.1, t["counts"], t["offsets"], t["used"], t["lse"], t["probs"], t["loss"]))


def balance_backward(rows, e, tx=F32, pad=0):
    m = (rows, e)
    return (dict(X=(m, tx), lse=((rows,), F32), counts=((e,), I32), used=((1,), I32), dloss=((1,), F32), dR=(m, tx)), dict(dX=(m, tx)), pad,
            lambda t: B.gemm_balance_backward(t["X"], t["lse"], t["counts"], t["used"], 0.1, t["dloss"], t["dR"], t["dX"]))


GRAD = B.GEMM_ACT_GRADIENT
CASES = {
    "linear one row": lambda: linear(1, 2048, 1024),
    "linear small tiles, split": lambda: linear(100, 2048, 512, path=1, bm=64, bn=128, split_k=4),
    "linear small tiles, gradient": lambda: linear(100, 512, 512, B.GEMM_FORM_NN, B.GEMM_ACT_GELU | GRAD, path=1, bm=128, bn=128, split_k=1),
    "linear two-SM tiles": lambda: linear(600, 512, 776, path=0, bm=256, bn=256, split_k=1),
    "linear two-SM tiles, gradient": lambda: linear(600, 512, 776, B.GEMM_FORM_NN, B.GEMM_ACT_GELU | GRAD, path=0, bm=256, bn=256, split_k=1),
    "linear weight gradient": lambda: linear(256, 700, 512, B.GEMM_FORM_TN, B.GEMM_ACT_NONE, F32),
    "linear unaligned": lambda: linear(300, 333, 401, pad=1),
    "activation": lambda: activation(3000, 512),
    "activation shifted": lambda: activation(3000, 501, 2),
    "activation few rows": lambda: activation(30, 640),
    "norm a CTA per row": lambda: norm(40, 776),
    "norm warps": lambda: norm(3000, 120),
    "norm a warp per row": lambda: norm(3000, 640),
    "norm ring": lambda: norm(3000, 1032),
    "norm unaligned": lambda: norm(3000, 401),
    "norm unaligned, pitch": lambda: norm(1000, 1001, F32, 2),
    "norm backward warps": lambda: norm_backward(3000, 120),
    "norm backward ring": lambda: norm_backward(3000, 1032),
    "norm backward unaligned": lambda: norm_backward(3000, 401, F32),
    "norm backward few rows": lambda: norm_backward(40, 1032),
    "norm backward long rows": lambda: norm_backward(600, 9000),
    "balance few rows": lambda: balance(40, 32),
    "balance one cluster": lambda: balance(900, 64),
    "balance many rows": lambda: balance(60000, 64),
    "balance odd": lambda: balance(30000, 33, 2, BF16),
    "balance backward": lambda: balance_backward(20000, 64),
    "balance backward few rows": lambda: balance_backward(40, 33, BF16),
}


def content(shape, dtype, g):
    if dtype == I32:
        return torch.randint(1, 8, shape, generator=g, device="cuda", dtype=I32)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


class Buffer:
    """A tensor of rows with a pitch in a buffer of whole 16-byte words."""

    def __init__(self, shape, dtype, pad):
        rows, cols = shape if len(shape) == 2 else (1, shape[0])
        pitch = cols + (pad if len(shape) == 2 and dtype != I32 else 0)
        n = rows * pitch
        self.all = torch.zeros((n + 15) // 16 * 16, dtype=dtype, device="cuda")
        view = self.all[:n].view(rows, pitch)[:, :cols]
        self.view = view if len(shape) == 2 else view[0]


@pytest.mark.parametrize("name", list(CASES))
def test_late_writes_are_waited_for(writer, name):  # noqa: F811
    ins, outs, pad, call = CASES[name]()
    g = torch.Generator(device="cuda")
    g.manual_seed(len(name))
    buffers = {n: Buffer(shape, dtype, pad) for n, (shape, dtype) in {**ins, **outs}.items()}
    views = {n: b.view for n, b in buffers.items()}
    good = {n: content(shape, dtype, g) for n, (shape, dtype) in ins.items()}
    if "rstd" in ins:
        good["rstd"] = good["rstd"].abs()
    for n in ins:
        views[n].copy_(good[n])
    call(views)
    want = {n: views[n].clone() for n in outs}
    stream = torch.cuda.current_stream()
    for late in buffers:
        src = buffers[late].all.clone()
        if late in outs:
            src.fill_(5)
        for rep in range(2):
            for n in buffers:
                if n in outs:
                    buffers[n].all.fill_(3)
                else:
                    views[n].copy_(good[n])
            buffers[late].all.zero_()
            torch.cuda.synchronize()
            assert writer.late_writer(buffers[late].all.data_ptr(), src.data_ptr(), src.numel() * src.element_size(), 50_000,
                                      stream.cuda_stream) == 0
            call(views)
            torch.cuda.synchronize()
            for n in outs:
                assert torch.equal(views[n], want[n]), (late, n, rep)
