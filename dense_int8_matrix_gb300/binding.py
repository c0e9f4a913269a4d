"""ctypes binding of libgemm_gb300.so (include/dense_int8_matrix.h).

Argument marshalling only: every step of the GEMM runs in the library's CUDA
kernels.  Functions carry the C names.  Device buffers may be passed as
torch CUDA tensors (checked for dtype, shape, contiguity and device) or as
raw integer addresses.  If the library is missing, the first call raises;
there is no fallback.
"""

from __future__ import annotations

import ctypes
import os

from . import build as _build

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_MISALIGNED = 2
GEMM_ERR_UNSUPPORTED_DEVICE = 3
GEMM_ERR_CUDA = 4
GEMM_ERR_OVERFLOW_RISK = 5
GEMM_ERR_TIMEOUT = 6

GEMM_PATH_TENSOR = 0
GEMM_PATH_SKINNY = 1
GEMM_DTYPE_I8 = 0
GEMM_DTYPE_BF16 = 1
GEMM_KERNEL_STAGE = 0
GEMM_KERNEL_TC = 1
GEMM_KERNEL_SKINNY = 2
GEMM_KERNEL_REQUANT = 3
GEMM_KERNEL_KINDS = 4
GEMM_OUT_BF16 = 1
GEMM_OUT_I8 = 2
GEMM_OUT_F32 = 3
GEMM_DTYPE_F32 = 2
GEMM_F8_E4M3 = 0
GEMM_F8_E5M2 = 1
GEMM_SCALE_ROWS = 0
GEMM_SCALE_BLOCKS = 1
GEMM_GROUP_NONE = 0
GEMM_GROUP_ROWS = 1
GEMM_GROUP_K = 2
GEMM_FORM_NT = 0
GEMM_FORM_NN = 1
GEMM_FORM_TN = 2
GEMM_ACT_NONE = 0
GEMM_ACT_RELU = 1
GEMM_ACT_GELU = 2
GEMM_ACT_GELU_TANH = 3
GEMM_ACT_SILU = 4
GEMM_ACT_GRADIENT = 16
GEMM_PLAN_LINEAR_VERSION = 1
GEMM_BALANCE_MAX_EXPERTS = 1024
GEMM_PLAN_F8_VERSION = 1
GEMM_F8_MAX_GROUPS = 1024
GEMM_NORM_MAX_D = 32768
GEMM_PLAN_VERSION = 2
GEMM_I8_MAX_K = 131071
GEMM_NOALLOC_SCRATCH_BYTES = 64 << 20

# every function the header declares
EXPORTED = (
    "gemm_i8_plan", "gemm_bf16_plan", "gemm_plan_for_sms", "gemm_i8_run", "gemm_bf16_run",
    "gemm_i8_run_host", "gemm_bf16_run_host", "gemm_device_error", "gemm_trace_begin",
    "gemm_trace_collect", "gemm_tc_kernel_info", "gemm_selftest_wait_timeout", "gemm_status_string",
    "gemm_i8_run_noalloc", "gemm_pool_usage", "gemm_i8_run_requant",
    "gemm_f8_plan", "gemm_f8_grouped_plan", "gemm_f8_plan_for_sms", "gemm_f8_run", "gemm_f8_grouped_run",
    "gemm_f8_quantize", "gemm_f8_quantize_cols", "gemm_f8_padded_k", "gemm_norm_f8", "gemm_norm_i8",
    "gemm_norm_backward", "gemm_bf16_linear_plan", "gemm_bf16_linear_plan_for_sms", "gemm_bf16_linear_run",
    "gemm_activation_backward", "gemm_layer_norm", "gemm_layer_norm_backward", "gemm_balance", "gemm_balance_backward",
)


class gemm_plan(ctypes.Structure):
    _fields_ = [
        ("version", ctypes.c_int32), ("path", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("num_sms", ctypes.c_int32),
        ("m", ctypes.c_int64), ("k", ctypes.c_int64), ("n", ctypes.c_int64),
        ("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("bk", ctypes.c_int32),
        ("stages", ctypes.c_int32), ("tiles", ctypes.c_int32), ("bpc", ctypes.c_int32),
        ("grid", ctypes.c_int32), ("waves", ctypes.c_int32), ("k_pitch", ctypes.c_int32),
        ("chunk_k", ctypes.c_int32), ("fallback", ctypes.c_int32), ("split_k", ctypes.c_int32),
        ("ratio", ctypes.c_double), ("workspace_bytes", ctypes.c_int64),
        ("split_from", ctypes.c_int32), ("a_on_chip", ctypes.c_int32),
        ("reserved", ctypes.c_int64 * 3),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_
                if not name.startswith("reserved")}


class gemm_plan_f8(ctypes.Structure):
    _fields_ = [
        ("version", ctypes.c_int32), ("path", ctypes.c_int32), ("num_sms", ctypes.c_int32),
        ("group_mode", ctypes.c_int32),
        ("m", ctypes.c_int64), ("k", ctypes.c_int64), ("n", ctypes.c_int64),
        ("groups", ctypes.c_int32), ("a_type", ctypes.c_int32), ("b_type", ctypes.c_int32),
        ("b_scale", ctypes.c_int32), ("bm", ctypes.c_int32), ("bn", ctypes.c_int32),
        ("split_k", ctypes.c_int32), ("reserved32", ctypes.c_int32),
        ("reserved", ctypes.c_int64 * 4),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_
                if not name.startswith("reserved")}


class gemm_plan_linear(ctypes.Structure):
    _fields_ = [
        ("version", ctypes.c_int32), ("path", ctypes.c_int32), ("num_sms", ctypes.c_int32),
        ("form", ctypes.c_int32),
        ("m", ctypes.c_int64), ("k", ctypes.c_int64), ("n", ctypes.c_int64),
        ("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("split_k", ctypes.c_int32), ("reserved32", ctypes.c_int32),
        ("reserved", ctypes.c_int64 * 4),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_
                if not name.startswith("reserved")}


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, _status_name(status)))


_lib = None


def _status_name(s: int) -> str:
    names = {0: "GEMM_OK", 1: "GEMM_ERR_INVALID_ARG", 2: "GEMM_ERR_MISALIGNED",
             3: "GEMM_ERR_UNSUPPORTED_DEVICE", 4: "GEMM_ERR_CUDA", 5: "GEMM_ERR_OVERFLOW_RISK",
             6: "GEMM_ERR_TIMEOUT"}
    return names.get(s, "status %d" % s)


def library_path() -> str:
    return _build.LIB_PATH


def load():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError("%s is not built (run __graft_entry__.build()); "
                           "the GEMM has no CPU fallback" % path)
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(gemm_plan)
    P8 = ctypes.POINTER(gemm_plan_f8)
    PL = ctypes.POINTER(gemm_plan_linear)
    i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
    sig = {
        "gemm_i8_plan": [i64, i64, i64, P],
        "gemm_bf16_plan": [i64, i64, i64, P],
        "gemm_plan_for_sms": [i32, i64, i64, i64, i32, P],
        "gemm_i8_run": [P, vp, vp, vp, vp],
        "gemm_bf16_run": [P, vp, vp, vp, vp],
        "gemm_i8_run_host": [P, vp, vp, vp, vp],
        "gemm_bf16_run_host": [P, vp, vp, vp, vp],
        "gemm_device_error": [vp, ctypes.POINTER(i32)],
        "gemm_trace_begin": [i32, i32],
        "gemm_trace_collect": [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(i32), ctypes.POINTER(i32)],
        "gemm_tc_kernel_info": [i32, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)],
        "gemm_selftest_wait_timeout": [i32, vp],
        "gemm_i8_run_noalloc": [P, vp, vp, vp, vp],
        "gemm_pool_usage": [ctypes.POINTER(i64), ctypes.POINTER(i64), i32],
        "gemm_i8_run_requant": [P, vp, vp, vp, vp, i32, vp, vp],
        "gemm_f8_plan": [i64, i64, i64, i32, i32, i32, P8],
        "gemm_f8_grouped_plan": [i32, i32, i64, i64, i64, i32, i32, i32, P8],
        "gemm_f8_plan_for_sms": [i32, i32, i64, i64, i64, i32, i32, i32, i32, P8],
        "gemm_f8_run": [P8, vp, i64, vp, vp, i64, vp, i32, vp, i64, vp],
        "gemm_f8_grouped_run": [P8, vp, i64, vp, vp, i64, vp, vp, i32, vp, i64, vp],
        "gemm_f8_quantize": [vp, i32, i64, i64, i64, i32, i32, vp, i64, vp, vp],
        "gemm_f8_quantize_cols": [vp, i32, i64, i64, i64, i32, vp, i32, vp, i64, vp, vp],
        "gemm_norm_f8": [vp, i64, vp, i64, vp, f32, i32, i64, i64, vp, i64, vp, vp, i64, vp, vp],
        "gemm_norm_i8": [vp, i64, vp, i64, vp, f32, i32, i64, i64, vp, i64, vp, vp, i64, vp, vp],
        "gemm_norm_backward": [vp, i64, vp, i64, vp, vp, vp, i64, i32, i64, i64, vp, i64, vp, vp],
        "gemm_bf16_linear_plan": [i32, i64, i64, i64, PL],
        "gemm_bf16_linear_plan_for_sms": [i32, i64, i64, i64, i32, PL],
        "gemm_bf16_linear_run": [PL, vp, i64, vp, i64, vp, i32, vp, i64, vp, i64, i32, vp, i64, vp],
        "gemm_activation_backward": [vp, i64, vp, i64, i32, i64, i64, vp, i64, vp, vp],
        "gemm_layer_norm": [vp, i64, vp, i64, vp, vp, f32, i32, i32, i64, i64, vp, i64, vp, vp, vp, i64, vp],
        "gemm_layer_norm_backward": [vp, i64, vp, i64, vp, vp, vp, vp, i64, i32, i32, i64, i64, vp, i64, vp, vp, vp],
        "gemm_balance": [vp, i64, i32, i64, i32, vp, i32, f32, vp, vp, vp, vp, vp, vp, vp],
        "gemm_balance_backward": [vp, i64, i32, i64, i32, vp, vp, vp, f32, vp, vp, i64, vp, i64, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.gemm_f8_padded_k.argtypes = [i64, i32]
    lib.gemm_f8_padded_k.restype = i64
    lib.gemm_status_string.argtypes = [ctypes.c_int]
    lib.gemm_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def gemm_status_string(status: int) -> str:
    return load().gemm_status_string(status).decode()


def _check(status: int, where: str):
    if status != GEMM_OK:
        raise GemmError(status, where)


# ------------------------------------------------------------------ plans --

def gemm_i8_plan(m: int, k: int, n: int) -> gemm_plan:
    p = gemm_plan()
    _check(load().gemm_i8_plan(m, k, n, ctypes.byref(p)), "gemm_i8_plan")
    return p


def gemm_bf16_plan(m: int, k: int, n: int) -> gemm_plan:
    p = gemm_plan()
    _check(load().gemm_bf16_plan(m, k, n, ctypes.byref(p)), "gemm_bf16_plan")
    return p


def gemm_plan_for_sms(dtype: int, m: int, k: int, n: int, num_sms: int) -> gemm_plan:
    p = gemm_plan()
    _check(load().gemm_plan_for_sms(dtype, m, k, n, num_sms, ctypes.byref(p)), "gemm_plan_for_sms")
    return p


# -------------------------------------------------------------------- run --

def _current_device() -> int:
    import torch
    return torch._C._cuda_getDevice()


def _addr(x, dtype=None, shape=None, device=True):
    """Address of a tensor (after checks) or an integer address as is.  The
    library works on the current device, so a CUDA tensor has to be there."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("expected a torch tensor or an integer address")
    if dtype is not None and x.dtype != dtype:
        raise TypeError("expected %s, got %s" % (dtype, x.dtype))
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError("expected shape %s, got %s" % (tuple(shape), tuple(x.shape)))
    if not x.is_contiguous():
        raise ValueError("tensor must be contiguous")
    if device and not x.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if device and x.get_device() != _current_device():
        raise ValueError("the tensor is on cuda:%d, the current device is cuda:%d" % (x.get_device(), _current_device()))
    if not device and x.is_cuda:
        raise ValueError("tensor must be in host memory")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        if not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream
        # the same handle without building a Stream object (0.4 us against 2.9)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def gemm_i8_run(plan: gemm_plan, A, Bt, C, stream=None) -> None:
    import torch
    m, k, n = plan.m, plan.k, plan.n
    st = load().gemm_i8_run(ctypes.byref(plan), _addr(A, torch.int8, (m, k)), _addr(Bt, torch.int8, (n, k)),
                            _addr(C, torch.int32, (m, n)), _stream(stream))
    _check(st, "gemm_i8_run")


def gemm_bf16_run(plan: gemm_plan, A, Bt, C, stream=None) -> None:
    import torch
    m, k, n = plan.m, plan.k, plan.n
    st = load().gemm_bf16_run(ctypes.byref(plan), _addr(A, torch.bfloat16, (m, k)),
                              _addr(Bt, torch.bfloat16, (n, k)), _addr(C, torch.float32, (m, n)),
                              _stream(stream))
    _check(st, "gemm_bf16_run")


def gemm_i8_run_noalloc(plan: gemm_plan, A, Bt, C, stream=None) -> None:
    """gemm_i8_run without device allocation (fixed 64 MiB static scratch)."""
    import torch
    m, k, n = plan.m, plan.k, plan.n
    st = load().gemm_i8_run_noalloc(ctypes.byref(plan), _addr(A, torch.int8, (m, k)),
                                    _addr(Bt, torch.int8, (n, k)), _addr(C, torch.int32, (m, n)),
                                    _stream(stream))
    _check(st, "gemm_i8_run_noalloc")


def gemm_i8_run_requant(plan: gemm_plan, A, Bt, row_scale, col_scale, D, out_type=None, stream=None) -> None:
    """D = q((float(A x B) * row_scale[i]) * col_scale[j]) with q = bfloat16
    (D a torch.bfloat16 tensor) or saturated int8 (D a torch.int8 tensor)."""
    import torch
    m, k, n = plan.m, plan.k, plan.n
    if out_type is None:
        out_type = GEMM_OUT_BF16 if isinstance(D, torch.Tensor) and D.dtype == torch.bfloat16 else GEMM_OUT_I8
    d_dtype = torch.bfloat16 if out_type == GEMM_OUT_BF16 else torch.int8
    st = load().gemm_i8_run_requant(ctypes.byref(plan), _addr(A, torch.int8, (m, k)), _addr(Bt, torch.int8, (n, k)),
                                    _addr(row_scale, torch.float32, (m,)), _addr(col_scale, torch.float32, (n,)),
                                    out_type, _addr(D, d_dtype, (m, n)), _stream(stream))
    _check(st, "gemm_i8_run_requant")


def gemm_i8_run_host(plan: gemm_plan, A, Bt, C, stream=None) -> None:
    import torch
    m, k, n = plan.m, plan.k, plan.n
    st = load().gemm_i8_run_host(ctypes.byref(plan), _addr(A, torch.int8, (m, k), device=False),
                                 _addr(Bt, torch.int8, (n, k), device=False),
                                 _addr(C, torch.int32, (m, n), device=False), _stream(stream))
    _check(st, "gemm_i8_run_host")


def gemm_bf16_run_host(plan: gemm_plan, A, Bt, C, stream=None) -> None:
    import torch
    m, k, n = plan.m, plan.k, plan.n
    st = load().gemm_bf16_run_host(ctypes.byref(plan), _addr(A, torch.bfloat16, (m, k), device=False),
                                   _addr(Bt, torch.bfloat16, (n, k), device=False),
                                   _addr(C, torch.float32, (m, n), device=False), _stream(stream))
    _check(st, "gemm_bf16_run_host")


def gemm_device_error(stream=None):
    """(status, code): GEMM_OK or GEMM_ERR_TIMEOUT with the stage that gave up."""
    code = ctypes.c_int32(0)
    st = load().gemm_device_error(_stream(stream), ctypes.byref(code))
    return st, code.value


def gemm_pool_usage(reset_high: bool = False):
    """(bytes the library's pool holds, most bytes in use at once since the
    last reset); reset_high restarts the second from the current use."""
    reserved = ctypes.c_int64(0)
    high = ctypes.c_int64(0)
    _check(load().gemm_pool_usage(ctypes.byref(reserved), ctypes.byref(high), 1 if reset_high else 0),
           "gemm_pool_usage")
    return reserved.value, high.value


def gemm_trace_begin(capacity: int, every: int = 1) -> None:
    _check(load().gemm_trace_begin(capacity, every), "gemm_trace_begin")


def gemm_trace_collect():
    """Per kind: (summed ms of the timed units, timed units, launches counted)."""
    ms = (ctypes.c_float * GEMM_KERNEL_KINDS)()
    timed = (ctypes.c_int32 * GEMM_KERNEL_KINDS)()
    cnt = (ctypes.c_int32 * GEMM_KERNEL_KINDS)()
    _check(load().gemm_trace_collect(ms, timed, cnt), "gemm_trace_collect")
    return list(ms), list(timed), list(cnt)


def gemm_tc_kernel_info(bm: int, bn: int, dtype: int):
    regs = ctypes.c_int32(0)
    occ = ctypes.c_int32(0)
    _check(load().gemm_tc_kernel_info(bm, bn, dtype, ctypes.byref(regs), ctypes.byref(occ)),
           "gemm_tc_kernel_info")
    return regs.value, occ.value


def gemm_selftest_wait_timeout(timeout_us: int, stream=None) -> None:
    _check(load().gemm_selftest_wait_timeout(timeout_us, _stream(stream)), "gemm_selftest_wait_timeout")


# ------------------------------------------------------- 8-bit operators --

def gemm_f8_plan(m: int, k: int, n: int, a_type: int = GEMM_F8_E4M3, b_type: int = GEMM_F8_E4M3,
                 b_scale: int = GEMM_SCALE_BLOCKS) -> gemm_plan_f8:
    p = gemm_plan_f8()
    _check(load().gemm_f8_plan(m, k, n, a_type, b_type, b_scale, ctypes.byref(p)), "gemm_f8_plan")
    return p


def gemm_f8_grouped_plan(group_mode: int, groups: int, m: int, k: int, n: int, a_type: int = GEMM_F8_E4M3,
                         b_type: int = GEMM_F8_E4M3, b_scale: int = GEMM_SCALE_BLOCKS) -> gemm_plan_f8:
    p = gemm_plan_f8()
    _check(load().gemm_f8_grouped_plan(group_mode, groups, m, k, n, a_type, b_type, b_scale, ctypes.byref(p)),
           "gemm_f8_grouped_plan")
    return p


def gemm_f8_plan_for_sms(group_mode: int, groups: int, m: int, k: int, n: int, num_sms: int,
                         a_type: int = GEMM_F8_E4M3, b_type: int = GEMM_F8_E4M3,
                         b_scale: int = GEMM_SCALE_BLOCKS) -> gemm_plan_f8:
    p = gemm_plan_f8()
    _check(load().gemm_f8_plan_for_sms(group_mode, groups, m, k, n, a_type, b_type, b_scale, num_sms,
                                       ctypes.byref(p)), "gemm_f8_plan_for_sms")
    return p


def gemm_f8_padded_k(rows: int, groups: int = 1) -> int:
    return load().gemm_f8_padded_k(rows, groups)


class _Torch:
    """What the calls below need of torch, looked up once: a small call is as
    long as its checks and its launch."""

    def __init__(self):
        import torch
        self.f32, self.bf16, self.i32, self.i8 = torch.float32, torch.bfloat16, torch.int32, torch.int8
        self.f8 = (torch.float8_e4m3fn, torch.float8_e5m2)   # by GEMM_F8_*
        self.f8_type = {d: i for i, d in enumerate(self.f8)}
        self.real_type = {torch.bfloat16: GEMM_DTYPE_BF16, torch.float32: GEMM_DTYPE_F32}
        self.out_type = {torch.bfloat16: GEMM_OUT_BF16, torch.float32: GEMM_OUT_F32}
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.current_device = torch._C._cuda_getDevice


_torch_names = None


def _torch():
    global _torch_names
    if _torch_names is None:
        _torch_names = _Torch()
    return _torch_names


def _type_of(x, types):
    found = types.get(x.dtype)
    if found is None:
        raise TypeError("expected %s, got %s" % (" or ".join(str(d) for d in types), x.dtype))
    return found


def _stream_of(dev, stream):
    """The CUDA stream handle for a call on tensors of device `dev`; by default
    its current stream.  The library works on the current device (its SMs, its
    scratch, its launches), so that is the only one whose tensors it takes."""
    if dev < 0:
        raise ValueError("tensor must be on a CUDA device")
    here = _torch_names.current_device()
    if dev != here:
        raise ValueError("the tensors are on cuda:%d, the current device is cuda:%d" % (dev, here))
    if stream is None:
        return _torch_names.raw_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _wrong(x, dtype, shape, dev):
    if x.dtype is not dtype:
        raise TypeError("expected %s, got %s" % (dtype, x.dtype))
    if x.shape != shape:
        raise ValueError("expected shape %s, got %s" % (tuple(shape), tuple(x.shape)))
    if x.get_device() < 0:
        raise ValueError("tensor must be on a CUDA device")
    if x.get_device() != dev:   # (dev itself is -1 if the first tensor is on the host)
        raise ValueError("the tensors of a call must be on one device: %d and %d" % (dev, x.get_device()))
    raise ValueError("tensor must be contiguous")


def _dense(x, dtype, shape, dev):
    """Address of a contiguous tensor of device `dev` (_stream_of checks dev)."""
    if x.dtype is not dtype or x.shape != shape or x.get_device() != dev or not x.is_contiguous():
        _wrong(x, dtype, shape, dev)
    return x.data_ptr()


def _matrix(x, dtype, shape, dev):
    """(address, row pitch) of a tensor of device `dev` whose rows are
    contiguous; the leading dimensions before the last two lie one after the
    other."""
    if x.dtype is not dtype or x.shape != shape or x.get_device() != dev:
        _wrong(x, dtype, shape, dev)
    stride = x.stride()
    cols = shape[-1]
    groups = shape[0] if len(shape) == 3 else 1
    if shape[-2] > 1:
        pitch = stride[-2]
    elif groups > 1:
        pitch = stride[0]
    else:   # one row: any pitch will do
        pitch = (cols + 15) // 16 * 16
    if (cols > 1 and stride[-1] != 1) or pitch < cols:
        raise ValueError("rows must be contiguous and must not overlap")
    if groups > 1 and stride[0] != pitch * shape[1]:
        raise ValueError("groups must lie one after the other")
    return x.data_ptr(), pitch


def _f8_run(plan, A, a_scale, Bt, b_scale, offsets, D, stream):
    lib, T = _lib or load(), _torch_names or _torch()
    m, k, n, g, mode = plan.m, plan.k, plan.n, plan.groups, plan.group_mode
    kb = (k + 127) // 128
    dev = A.get_device()
    a, lda = _matrix(A, T.f8[plan.a_type], (m, k), dev)
    rows = mode == GEMM_GROUP_ROWS
    b, ldb = _matrix(Bt, T.f8[plan.b_type], (g, n, k) if rows else (n, k), dev)
    if plan.b_scale == GEMM_SCALE_BLOCKS:
        sb = _dense(b_scale, T.f32, (g, (n + 127) // 128, kb) if rows else ((n + 127) // 128, kb), dev)
    else:
        sb = _dense(b_scale, T.f32, (kb, g * n) if rows else (kb, n), dev)
    sa = _dense(a_scale, T.f32, (kb, m), dev)
    out = _type_of(D, T.out_type)
    d, ldd = _matrix(D, D.dtype, (g, m, n) if mode == GEMM_GROUP_K else (m, n), dev)
    s = _stream_of(dev, stream)
    if offsets is None:
        return lib.gemm_f8_run(plan, a, lda, sa, b, ldb, sb, out, d, ldd, s)
    off = _dense(offsets, T.i32, (g + 1,), dev)
    return lib.gemm_f8_grouped_run(plan, a, lda, sa, b, ldb, sb, off, out, d, ldd, s)


def gemm_f8_run(plan: gemm_plan_f8, A, a_scale, Bt, b_scale, D, stream=None) -> None:
    """D (m x n, bfloat16 or fp32) = A x B for FP8 tensors A (m x k) and Bt
    (n x k) with fp32 scales: a_scale (ceil(k/128), m); b_scale
    (ceil(n/128), ceil(k/128)), or (ceil(k/128), n) for a plan with
    GEMM_SCALE_ROWS.  Rows may have a pitch (a multiple of 16 for A and Bt)."""
    st = _f8_run(plan, A, a_scale, Bt, b_scale, None, D, stream)
    if st:
        _check(st, "gemm_f8_run")


def gemm_f8_grouped_run(plan: gemm_plan_f8, A, a_scale, Bt, b_scale, offsets, D, stream=None) -> None:
    """The grouped product.  GEMM_GROUP_ROWS: Bt (groups, n, k), b_scale
    (groups, ceil(n/128), ceil(k/128)); rows offsets[g]:offsets[g+1] of A and
    D belong to group g.  GEMM_GROUP_K: A (m, k), Bt (n, k) from
    gemm_f8_quantize_cols with the same offsets, D (groups, m, n).  offsets:
    groups + 1 int32 on the GPU."""
    if offsets is None:
        raise TypeError("offsets are needed")
    st = _f8_run(plan, A, a_scale, Bt, b_scale, offsets, D, stream)
    if st:
        _check(st, "gemm_f8_grouped_run")


def gemm_f8_quantize(X, Q, scale, scale_mode: int = GEMM_SCALE_ROWS, stream=None) -> None:
    """Q (float8, like X) and its scales from X (rows x cols, bfloat16 or
    fp32): scale (ceil(cols/128), rows), or (ceil(rows/128), ceil(cols/128))
    for GEMM_SCALE_BLOCKS."""
    lib, T = _lib or load(), _torch_names or _torch()
    rows, cols = shape = X.shape
    dev = X.get_device()
    x, ldx = _matrix(X, X.dtype, shape, dev)
    q, ldq = _matrix(Q, Q.dtype, shape, dev)
    kb = (cols + 127) // 128
    sshape = (kb, rows) if scale_mode == GEMM_SCALE_ROWS else ((rows + 127) // 128, kb)
    st = lib.gemm_f8_quantize(x, _type_of(X, T.real_type), rows, cols, ldx, _type_of(Q, T.f8_type), scale_mode, q, ldq,
                              _dense(scale, T.f32, sshape, dev), _stream_of(dev, stream))
    if st:
        _check(st, "gemm_f8_quantize")


def gemm_f8_quantize_cols(X, Q, scale, offsets=None, stream=None) -> None:
    """Q (cols x gemm_f8_padded_k(rows, groups), float8) = X^T quantised in
    blocks of 128 rows of each group, scale (padded_k / 128, cols).  offsets:
    groups + 1 int32 on the GPU, None for one group of all rows."""
    lib, T = _lib or load(), _torch_names or _torch()
    rows, cols = shape = X.shape
    dev = X.get_device()
    groups = 1 if offsets is None else offsets.shape[0] - 1
    kp = (rows + 127 * groups) // 128 * 128
    x, ldx = _matrix(X, X.dtype, shape, dev)
    q, ldq = _matrix(Q, Q.dtype, (cols, kp), dev)
    off = None if offsets is None else _dense(offsets, T.i32, (groups + 1,), dev)
    st = lib.gemm_f8_quantize_cols(x, _type_of(X, T.real_type), rows, cols, ldx, _type_of(Q, T.f8_type), off, groups, q,
                                   ldq, _dense(scale, T.f32, (kp // 128, cols), dev), _stream_of(dev, stream))
    if st:
        _check(st, "gemm_f8_quantize_cols")


def _norm(call, name, X, R, W, eps, H, rstd, Q, q_dtype, scale, scale_shape, stream):
    T = _torch_names
    rows, d = shape = X.shape
    dev = X.get_device()
    x, ldx = _matrix(X, X.dtype, shape, dev)
    r, ldr = (None, 0) if R is None else _matrix(R, X.dtype, shape, dev)
    h, ldh = (None, 0) if H is None else _matrix(H, X.dtype, shape, dev)
    q, ldq = _matrix(Q, q_dtype, shape, dev)
    st = call(x, ldx, r, ldr, _dense(W, T.f32, (d,), dev), eps, _type_of(X, T.real_type), rows, d, h, ldh,
              None if rstd is None else _dense(rstd, T.f32, (rows,), dev), q, ldq, _dense(scale, T.f32, scale_shape, dev),
              _stream_of(dev, stream))
    if st:
        _check(st, name)


def gemm_norm_f8(X, R, W, eps, H, rstd, Q, scale, stream=None) -> None:
    """h = X + R (kept in H), rstd, and y = h * rstd * W as e4m3 Q with scale
    (ceil(d/128), rows).  R, H and rstd may be None (H only without R)."""
    lib, T = _lib or load(), _torch_names or _torch()
    rows, d = X.shape
    _norm(lib.gemm_norm_f8, "gemm_norm_f8", X, R, W, eps, H, rstd, Q, T.f8[0], scale, ((d + 127) // 128, rows), stream)


def gemm_norm_i8(X, R, W, eps, H, rstd, Q, row_scale, stream=None) -> None:
    """As gemm_norm_f8 with int8 Q and one scale per row."""
    lib, T = _lib or load(), _torch_names or _torch()
    _norm(lib.gemm_norm_i8, "gemm_norm_i8", X, R, W, eps, H, rstd, Q, T.i8, row_scale, (X.shape[0],), stream)


def gemm_norm_backward(dY, H, W, rstd, dR, dX, dW, stream=None) -> None:
    """dX (the gradient of h) and dW from dY, the gradient of y; dR (may be
    None) is the gradient that reaches h as the residual, dW may be None."""
    lib, T = _lib or load(), _torch_names or _torch()
    rows, d = shape = dY.shape
    dt, dev = dY.dtype, dY.get_device()
    dy, lddy = _matrix(dY, dt, shape, dev)
    h, ldh = _matrix(H, dt, shape, dev)
    r, lddr = (None, 0) if dR is None else _matrix(dR, dt, shape, dev)
    dx, lddx = _matrix(dX, dt, shape, dev)
    st = lib.gemm_norm_backward(dy, lddy, h, ldh, _dense(W, T.f32, (d,), dev), _dense(rstd, T.f32, (rows,), dev), r, lddr,
                                _type_of(dY, T.real_type), rows, d, dx, lddx,
                                None if dW is None else _dense(dW, T.f32, (d,), dev), _stream_of(dev, stream))
    if st:
        _check(st, "gemm_norm_backward")


# ------------------------------------------------- bfloat16 layer operators --

def gemm_bf16_linear_plan(m: int, k: int, n: int, form: int = GEMM_FORM_NT) -> gemm_plan_linear:
    p = gemm_plan_linear()
    _check(load().gemm_bf16_linear_plan(form, m, k, n, ctypes.byref(p)), "gemm_bf16_linear_plan")
    return p


def gemm_bf16_linear_plan_for_sms(m: int, k: int, n: int, num_sms: int, form: int = GEMM_FORM_NT) -> gemm_plan_linear:
    p = gemm_plan_linear()
    _check(load().gemm_bf16_linear_plan_for_sms(form, m, k, n, num_sms, ctypes.byref(p)), "gemm_bf16_linear_plan_for_sms")
    return p


def _optional(x, dtype, shape, dev):
    return None if x is None else _dense(x, dtype, shape, dev)


def _optional_matrix(x, dtype, shape, dev):
    return (None, 0) if x is None else _matrix(x, dtype, shape, dev)


def gemm_bf16_linear_run(plan: gemm_plan_linear, A, B, D, bias=None, activation: int = GEMM_ACT_NONE, Z=None,
                         residual=None, stream=None) -> None:
    """D (m x n, bfloat16 or fp32) = act(A x B + bias) + residual, or with
    activation | GEMM_ACT_GRADIENT (A x B + bias) * act'(Z) + residual.  A, B:
    bfloat16, (m, k) and (n, k) for a plan of GEMM_FORM_NT, (m, k) and (k, n)
    for GEMM_FORM_NN, (k, m) and (k, n) for GEMM_FORM_TN.  bias: fp32 (n,); Z:
    bfloat16 (m, n), written without the gradient (A x B + bias) and read with
    it; residual: like D, may be D.  Rows may have a pitch."""
    lib, T = _lib or load(), _torch_names or _torch()
    m, k, n, form = plan.m, plan.k, plan.n, plan.form
    dev = A.get_device()
    a, lda = _matrix(A, T.bf16, (k, m) if form == GEMM_FORM_TN else (m, k), dev)
    b, ldb = _matrix(B, T.bf16, (n, k) if form == GEMM_FORM_NT else (k, n), dev)
    out = _type_of(D, T.out_type)
    d, ldd = _matrix(D, D.dtype, (m, n), dev)
    z, ldz = _optional_matrix(Z, T.bf16, (m, n), dev)
    r, ldr = _optional_matrix(residual, D.dtype, (m, n), dev)
    st = lib.gemm_bf16_linear_run(plan, a, lda, b, ldb, _optional(bias, T.f32, (n,), dev), activation, z, ldz, r, ldr, out,
                                  d, ldd, _stream_of(dev, stream))
    if st:
        _check(st, "gemm_bf16_linear_run")


def gemm_activation_backward(dY, Z, activation, dZ, dbias, stream=None) -> None:
    """dZ = dY * act'(Z) (bfloat16, may be dY or Z) and dbias (fp32, (cols,))
    = its sums over the rows; either may be None, Z for GEMM_ACT_NONE too."""
    lib, T = _lib or load(), _torch_names or _torch()
    rows, cols = shape = dY.shape
    dev = dY.get_device()
    y, lddy = _matrix(dY, T.bf16, shape, dev)
    z, ldz = _optional_matrix(Z, T.bf16, shape, dev)
    o, lddz = _optional_matrix(dZ, T.bf16, shape, dev)
    st = lib.gemm_activation_backward(y, lddy, z, ldz, activation, rows, cols, o, lddz, _optional(dbias, T.f32, (cols,), dev),
                                      _stream_of(dev, stream))
    if st:
        _check(st, "gemm_activation_backward")


def gemm_layer_norm(X, R, W, bias, eps, H, mean, rstd, Y, stream=None) -> None:
    """h = X + R (kept in H), mean and rstd of its rows, and Y (bfloat16 or
    fp32) = (h - mean) * rstd * W + bias.  R, bias, H (only without R), mean
    and rstd may be None."""
    lib, T = _lib or load(), _torch_names or _torch()
    rows, d = shape = X.shape
    dt, dev = X.dtype, X.get_device()
    x, ldx = _matrix(X, dt, shape, dev)
    r, ldr = _optional_matrix(R, dt, shape, dev)
    h, ldh = _optional_matrix(H, dt, shape, dev)
    y, ldy = _matrix(Y, Y.dtype, shape, dev)
    st = lib.gemm_layer_norm(x, ldx, r, ldr, _dense(W, T.f32, (d,), dev), _optional(bias, T.f32, (d,), dev), eps,
                             _type_of(X, T.real_type), _type_of(Y, T.real_type), rows, d, h, ldh,
                             _optional(mean, T.f32, (rows,), dev), _optional(rstd, T.f32, (rows,), dev), y, ldy,
                             _stream_of(dev, stream))
    if st:
        _check(st, "gemm_layer_norm")


def gemm_layer_norm_backward(dY, H, W, mean, rstd, dR, dX, dW, dbias, stream=None) -> None:
    """dX (the gradient of h, like H), dW and dbias (fp32) from dY, the
    gradient of Y; dR (may be None) is the gradient that reaches h as the
    residual; dW and dbias may be None."""
    lib, T = _lib or load(), _torch_names or _torch()
    rows, d = shape = H.shape
    dt, dev = H.dtype, H.get_device()
    dy, lddy = _matrix(dY, dY.dtype, shape, dev)
    h, ldh = _matrix(H, dt, shape, dev)
    r, lddr = _optional_matrix(dR, dt, shape, dev)
    dx, lddx = _matrix(dX, dt, shape, dev)
    st = lib.gemm_layer_norm_backward(dy, lddy, h, ldh, _dense(W, T.f32, (d,), dev), _dense(mean, T.f32, (rows,), dev),
                                      _dense(rstd, T.f32, (rows,), dev), r, lddr, _type_of(H, T.real_type),
                                      _type_of(dY, T.real_type), rows, d, dx, lddx, _optional(dW, T.f32, (d,), dev),
                                      _optional(dbias, T.f32, (d,), dev), _stream_of(dev, stream))
    if st:
        _check(st, "gemm_layer_norm_backward")


def gemm_balance(X, index, coef, counts, offsets, used, lse, probs, loss, stream=None) -> None:
    """Balance loss (fp32, (1,)) of the logits X (rows x experts, bfloat16 or
    fp32) and the experts chosen for each row, index (rows x top_k, int32; what
    lies outside [0, experts) is not taken): counts (experts,), offsets
    (experts + 1,; may be None) and used (1,) int32, lse (rows,) and probs
    (experts,) fp32."""
    lib, T = _lib or load(), _torch_names or _torch()
    rows, experts = shape = X.shape
    dev = X.get_device()
    x, ldx = _matrix(X, X.dtype, shape, dev)
    top_k = index.shape[-1]
    st = lib.gemm_balance(x, ldx, _type_of(X, T.real_type), rows, experts, _dense(index, T.i32, (rows, top_k), dev), top_k,
                          coef, _dense(counts, T.i32, (experts,), dev), _optional(offsets, T.i32, (experts + 1,), dev),
                          _dense(used, T.i32, (1,), dev), _dense(lse, T.f32, (rows,), dev),
                          _dense(probs, T.f32, (experts,), dev), _dense(loss, T.f32, (1,), dev), _stream_of(dev, stream))
    if st:
        _check(st, "gemm_balance")


def gemm_balance_backward(X, lse, counts, used, coef, dloss, dR, dX, stream=None) -> None:
    """dX (like X) = dR + the gradient of gemm_balance's loss times dloss
    (fp32, (1,)), from lse, counts and used as that call wrote them; dR may be
    None, or dX itself."""
    lib, T = _lib or load(), _torch_names or _torch()
    rows, experts = shape = X.shape
    dt, dev = X.dtype, X.get_device()
    x, ldx = _matrix(X, dt, shape, dev)
    r, lddr = _optional_matrix(dR, dt, shape, dev)
    dx, lddx = _matrix(dX, dt, shape, dev)
    st = lib.gemm_balance_backward(x, ldx, _type_of(X, T.real_type), rows, experts, _dense(lse, T.f32, (rows,), dev),
                                   _dense(counts, T.i32, (experts,), dev), _dense(used, T.i32, (1,), dev), coef,
                                   _dense(dloss, T.f32, (1,), dev), r, lddr, dx, lddx, _stream_of(dev, stream))
    if st:
        _check(st, "gemm_balance_backward")


# ------------------------------------------------------------ convenience --

def matmul_i8(A, Bt, out=None, stream=None):
    """int32 C = A x B for int8 CUDA tensors A (m x k) and Bt (n x k)."""
    import torch
    m, k = A.shape
    n = Bt.shape[0]
    plan = gemm_i8_plan(m, k, n)
    if out is None:
        out = torch.empty((m, n), dtype=torch.int32, device=A.device)
    gemm_i8_run(plan, A, Bt, out, stream)
    return out


def matmul_bf16(A, Bt, out=None, stream=None):
    """fp32 C = A x B for bf16 CUDA tensors A (m x k) and Bt (n x k)."""
    import torch
    m, k = A.shape
    n = Bt.shape[0]
    plan = gemm_bf16_plan(m, k, n)
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=A.device)
    gemm_bf16_run(plan, A, Bt, out, stream)
    return out
