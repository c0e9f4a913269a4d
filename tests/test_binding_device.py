"""The binding takes the tensors of a call only from the current device, on
which the library launches: host tensors that say they are on a CUDA device, a
stand-in for the device query and one for the library show it without a GPU."""

import types

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B

F8, BF16, F32, I32, I8 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32, torch.int8


class Placed(torch.Tensor):
    """A host tensor that names a CUDA device."""

    is_cuda = True

    def get_device(self):
        return self.device_index


def on(dev, *shape, dtype=F32):
    x = torch.zeros(*shape, dtype=dtype).as_subclass(Placed)
    x.device_index = dev
    return x


@pytest.fixture
def calls(monkeypatch):
    """What reaches the library; device 0 is current, and every device's
    default stream has the handle 0."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: made.append(name) or 0

    names = types.SimpleNamespace(**vars(B._torch()))
    names.current_device = lambda: 0
    names.raw_stream = lambda dev: 0
    monkeypatch.setattr(B, "_torch_names", names)
    monkeypatch.setattr(B, "_lib", Library())
    return made


def f8_plan(mode, g):
    p = B.gemm_plan_f8()
    p.m, p.k, p.n, p.groups, p.group_mode, p.b_scale = 64, 256, 128, g, mode, B.GEMM_SCALE_BLOCKS
    if mode == B.GEMM_GROUP_K:
        p.b_scale = B.GEMM_SCALE_ROWS
    return p


# each call: a function of its tensors, and the tensors' shapes and types in order
CALLS = {
    "gemm_f8_run": (
        lambda a, sa, b, sb, d: B.gemm_f8_run(f8_plan(B.GEMM_GROUP_NONE, 1), a, sa, b, sb, d),
        [((64, 256), F8), ((2, 64), F32), ((128, 256), F8), ((1, 2), F32), ((64, 128), BF16)]),
    "gemm_f8_grouped_run": (
        lambda a, sa, b, sb, off, d: B.gemm_f8_grouped_run(f8_plan(B.GEMM_GROUP_ROWS, 3), a, sa, b, sb, off, d),
        [((64, 256), F8), ((2, 64), F32), ((3, 128, 256), F8), ((3, 1, 2), F32), ((4,), I32), ((64, 128), BF16)]),
    "gemm_f8_grouped_run over K": (
        lambda a, sa, b, sb, off, d: B.gemm_f8_grouped_run(f8_plan(B.GEMM_GROUP_K, 3), a, sa, b, sb, off, d),
        [((64, 256), F8), ((2, 64), F32), ((128, 256), F8), ((2, 128), F32), ((4,), I32), ((3, 64, 128), F32)]),
    "gemm_f8_quantize": (
        lambda x, q, s: B.gemm_f8_quantize(x, q, s), [((40, 256), BF16), ((40, 256), F8), ((2, 40), F32)]),
    "gemm_f8_quantize_cols": (
        lambda x, q, s, off: B.gemm_f8_quantize_cols(x, q, s, off),
        [((40, 48), BF16), ((48, 384), F8), ((3, 48), F32), ((4,), I32)]),
    "gemm_norm_f8": (
        lambda x, r, w, h, rstd, q, s: B.gemm_norm_f8(x, r, w, 1e-6, h, rstd, q, s),
        [((5, 256), BF16), ((5, 256), BF16), ((256,), F32), ((5, 256), BF16), ((5,), F32), ((5, 256), F8), ((2, 5), F32)]),
    "gemm_norm_i8": (
        lambda x, r, w, h, rstd, q, s: B.gemm_norm_i8(x, r, w, 1e-6, h, rstd, q, s),
        [((5, 256), BF16), ((5, 256), BF16), ((256,), F32), ((5, 256), BF16), ((5,), F32), ((5, 256), torch.int8), ((5,), F32)]),
    "gemm_norm_backward": (
        lambda dy, h, w, rstd, dr, dx, dw: B.gemm_norm_backward(dy, h, w, rstd, dr, dx, dw),
        [((5, 256), F32), ((5, 256), F32), ((256,), F32), ((5,), F32), ((5, 256), F32), ((5, 256), F32), ((256,), F32)]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_only_tensors_of_the_current_device_reach_the_library(name, calls):
    call, operands = CALLS[name]

    def tensors(devs):
        return [on(d, *shape, dtype=dtype) for d, (shape, dtype) in zip(devs, operands)]

    n = len(operands)
    call(*tensors([0] * n))
    assert len(calls) == 1 and name.startswith(calls[0])
    with pytest.raises(ValueError, match="current device"):   # all on the other device
        call(*tensors([1] * n))
    for i in range(n):   # one of them there, or on the host
        for dev in (1, -1):
            devs = [0] * n
            devs[i] = dev
            with pytest.raises(ValueError, match="device"):
                call(*tensors(devs))
    with pytest.raises(ValueError, match="CUDA device"):
        call(*tensors([-1] * n))
    assert len(calls) == 1, "a refused call reached the library"


def plan(m, k, n):
    p = B.gemm_plan()
    p.m, p.k, p.n = m, k, n
    return p


OLDER = {
    "gemm_i8_run": (lambda a, b, c: B.gemm_i8_run(plan(4, 32, 8), a, b, c, stream=7), [(4, 32, I8), (8, 32, I8), (4, 8, I32)]),
    "gemm_bf16_run": (lambda a, b, c: B.gemm_bf16_run(plan(4, 32, 8), a, b, c, stream=7),
                      [(4, 32, BF16), (8, 32, BF16), (4, 8, F32)]),
    "gemm_i8_run_noalloc": (lambda a, b, c: B.gemm_i8_run_noalloc(plan(4, 32, 8), a, b, c, stream=7),
                            [(4, 32, I8), (8, 32, I8), (4, 8, I32)]),
    "gemm_i8_run_requant": (lambda a, b, r, s, d: B.gemm_i8_run_requant(plan(4, 32, 8), a, b, r, s, d, stream=7),
                            [(4, 32, I8), (8, 32, I8), (4, F32), (8, F32), (4, 8, BF16)]),
}


@pytest.mark.parametrize("name", list(OLDER))
def test_the_int8_and_bf16_products_take_the_current_device_only(name, calls, monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    call, operands = OLDER[name]
    n = len(operands)

    def tensors(devs):
        return [on(d, *o[:-1], dtype=o[-1]) for d, o in zip(devs, operands)]

    call(*tensors([0] * n))
    assert calls == [name]
    for i in range(n):
        devs = [0] * n
        devs[i] = 1
        with pytest.raises(ValueError, match="current device"):
            call(*tensors(devs))
    with pytest.raises(ValueError, match="current device"):
        call(*tensors([1] * n))
    assert calls == [name]
