"""64-bit references of the bfloat16 layer's operators and seeded inputs for
their tests (torch on the CPU; none of the library's code)."""

from __future__ import annotations

import math

import torch

from dense_int8_matrix_gb300 import binding as B

BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}   # of a rounding, relative to the value
ACTS = {"none": B.GEMM_ACT_NONE, "relu": B.GEMM_ACT_RELU, "gelu": B.GEMM_ACT_GELU, "gelu_tanh": B.GEMM_ACT_GELU_TANH,
        "silu": B.GEMM_ACT_SILU}


def gen(seed: int) -> torch.Generator:
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


def whole(shape, seed, most=8):
    """Whole numbers in [-most, most] as bfloat16: products and sums are exact."""
    return torch.randint(-most, most + 1, shape, generator=gen(seed)).to(BF16)


def normal(shape, seed, scale=1.0, dtype=BF16):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(dtype)


def act(name, v):
    if name == "relu":
        return v.clamp(min=0)
    if name == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        # (1 + tanh(u)) / 2 = 1 / (1 + exp(-2u)), which does not cancel in the left tail
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if name == "silu":
        return v * torch.sigmoid(v)
    return v


def slope(name, z):
    """The derivative by autograd, in 64 bits."""
    z = z.double().clone().requires_grad_(True)
    with torch.enable_grad():
        if name == "relu":
            return (z > 0).double().detach()
        return torch.autograd.grad(act(name, z).sum(), z)[0]


def operands(form, m, k, n, make):
    """A and B as the form stores them, and the m x k and k x n matrices."""
    a, b = make((m, k), 1), make((k, n), 2)
    A = a.T.contiguous() if form == B.GEMM_FORM_TN else a
    Bm = b.T.contiguous() if form == B.GEMM_FORM_NT else b
    return A, Bm, a.double(), b.double()


def padded(x, pad, at=0, fill=float("nan")):
    """x on the GPU as a view whose rows start `at` elements into a pitch of
    cols + pad, `fill` around it; and the whole buffer."""
    buf = torch.full((x.shape[0] * (x.shape[1] + pad) + at,), fill, dtype=x.dtype, device="cuda")
    view = buf[at:].view(x.shape[0], x.shape[1] + pad)[:, :x.shape[1]]
    view.copy_(x)
    return view, buf


def outside(buf, view):
    """The buffer's values that are not the view's."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    at = (view.data_ptr() - buf.data_ptr()) // buf.element_size()
    idx = at + torch.arange(view.shape[0], device=buf.device)[:, None] * view.stride(0) + torch.arange(view.shape[1], device=buf.device)
    mask[idx.flatten()] = False
    return buf[mask]


def layer_norm(x, r, w, b, eps, dtype):
    h = x if r is None else (x.double() + r.double()).to(F32).to(dtype)
    hd = h.double()
    mean = hd.mean(1)
    c = hd - mean[:, None]
    var = c.square().mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    y = c * rstd[:, None] * w.double()
    return h, mean, var, rstd, y if b is None else y + b.double()


def layer_norm_backward(dy, h, w, mean, rstd, dr):
    """dX, dW, db and the magnitudes that their errors go by."""
    dy, w, mean, rstd = dy.double(), w.double(), mean.double()[:, None], rstd.double()[:, None]
    xhat = (h.double() - mean) * rstd
    g = dy * w
    mg, mx = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = rstd * (g - mg - xhat * mx)
    size = rstd.abs() * (g.abs() + g.abs().mean(1, keepdim=True) + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    if dr is not None:
        dx, size = dx + dr.double(), size + dr.double().abs()
    return dx, (dy * xhat).sum(0), dy.sum(0), size, (dy * xhat).abs().sum(0), dy.abs().sum(0)


def balance(x, index, coef):
    """counts, offsets, used, lse, probs, loss and p, f, T for the gradient."""
    rows, e = x.shape
    taken = (index >= 0) & (index < e)
    used = taken.any(1)
    counts = torch.bincount(index[taken].long(), minlength=e)
    xd = x.double()
    lse = torch.logsumexp(xd, 1)
    dead = torch.isneginf(lse)
    # (not exp(x - lse): next to logits of the type's lowest value log(E) vanishes)
    p = torch.where((used & ~dead)[:, None], torch.softmax(torch.where(dead[:, None], 0.0, xd), 1), 0.0)
    lse = torch.where(used, lse, math.inf)
    t = int(used.sum())
    probs = p.sum(0) / max(t, 1)
    f = counts.double() / max(int(counts.sum()), 1)
    loss = coef * e * (f * probs).sum()
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    return counts, offsets, t, lse, probs, loss, p, f


def balance_gradient(p, f, t, coef, dloss, dr):
    e = p.shape[1]
    mix = (p * f).sum(1, keepdim=True)
    scale = dloss * coef * e / max(t, 1)
    d, size = scale * p * (f - mix), abs(scale) * p * (f + mix)
    return (d, size) if dr is None else (d + dr.double(), size + dr.double().abs())
