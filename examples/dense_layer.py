"""One training step of a feed-forward layer on the library's bfloat16 operators.

    out = h + W2 gelu(W1 norm(h) + b1) + b2,   h = x + r,   norm a layer norm

Forward: gemm_layer_norm adds the residual and normalises; two products with
bias, the first with the activation (and what it was applied to, kept for the
backward), the second with the residual in its epilogue.  Backward: the
gradient of a product's weights is a product over the rows (GEMM_FORM_TN), that
of its input one with the weights as they lie (GEMM_FORM_NN), through the
activation where there is one; gemm_activation_backward sums the biases'
gradients; gemm_layer_norm_backward takes the residual's.  Weights are bfloat16,
biases, the norm's weights and all their gradients fp32.  `python
examples/dense_layer.py` compares the step with the same layer in fp32 torch.
"""

from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from dense_int8_matrix_gb300 import binding as B  # noqa: E402

EPS = 1e-5
NAMES = ("out", "dx", "dnorm_w", "dnorm_b", "dw1", "db1", "dw2", "db2")


def product(form, a, b, dtype=torch.bfloat16, **more):
    """a b^T (GEMM_FORM_NT), a b (GEMM_FORM_NN) or a^T b (GEMM_FORM_TN)."""
    m, k = a.shape[::-1] if form == B.GEMM_FORM_TN else a.shape
    n = b.shape[0] if form == B.GEMM_FORM_NT else b.shape[1]
    out = torch.empty(m, n, dtype=dtype, device=a.device)
    B.gemm_bf16_linear_run(B.gemm_bf16_linear_plan(m, k, n, form), a, b, out, **more)
    return out


def column_sums(dy):
    out = torch.empty(dy.shape[1], device=dy.device)
    B.gemm_activation_backward(dy, None, B.GEMM_ACT_NONE, None, out)
    return out


def step(x, r, norm_w, norm_b, w1, b1, w2, b2, d_out):
    """Forward and backward.  x, r, d_out: (rows, d), w1: (ff, d), w2: (d, ff)
    bfloat16; norm_w, norm_b, b2: (d,), b1: (ff,) fp32.  Returns what NAMES says,
    dx being the gradient of x and of r."""
    rows, d = x.shape
    h, y = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=x.device), torch.empty(rows, device=x.device)
    B.gemm_layer_norm(x, r, norm_w, norm_b, EPS, h, mean, rstd, y)
    z = torch.empty(rows, w1.shape[0], dtype=x.dtype, device=x.device)
    a = product(B.GEMM_FORM_NT, y, w1, bias=b1, activation=B.GEMM_ACT_GELU, Z=z)
    out = product(B.GEMM_FORM_NT, a, w2, bias=b2, residual=h)

    dw2, db2 = product(B.GEMM_FORM_TN, d_out, a, torch.float32), column_sums(d_out)
    dz = product(B.GEMM_FORM_NN, d_out, w2, activation=B.GEMM_ACT_GELU | B.GEMM_ACT_GRADIENT, Z=z)
    dw1, db1 = product(B.GEMM_FORM_TN, dz, y, torch.float32), column_sums(dz)
    dy = product(B.GEMM_FORM_NN, dz, w1)
    dx, dnw, dnb = torch.empty_like(x), torch.empty_like(norm_w), torch.empty_like(norm_b)
    B.gemm_layer_norm_backward(dy, h, norm_w, mean, rstd, d_out, dx, dnw, dnb)
    return out, dx, dnw, dnb, dw1, db1, dw2, db2


def plain_step(x, r, norm_w, norm_b, w1, b1, w2, b2, d_out, dtype=torch.float32):
    """The same layer in torch with autograd, in `dtype`."""
    h0 = (x.to(dtype) + r.to(dtype)).to(x.dtype)
    h, nw, nb, a1, c1, a2, c2 = (t.detach().to(dtype).requires_grad_(True) for t in (h0, norm_w, norm_b, w1, b1, w2, b2))
    y = torch.nn.functional.layer_norm(h, h.shape[1:], nw, nb, EPS)
    out = h + torch.nn.functional.gelu(y @ a1.T + c1) @ a2.T + c2
    out.backward(d_out.to(dtype))
    return out.detach(), h.grad, nw.grad, nb.grad, a1.grad, c1.grad, a2.grad, c2.grad


def inputs(rows, d, ff, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf16 = torch.bfloat16
    return (rand(rows, d).to(bf16), rand(rows, d).to(bf16), 1 + 0.1 * rand(d), 0.1 * rand(d),
            (rand(ff, d) / d ** 0.5).to(bf16), 0.1 * rand(ff), (rand(d, ff) / ff ** 0.5).to(bf16), 0.1 * rand(d),
            (0.1 * rand(rows, d)).to(bf16))


def compare(rows=1000, d=512, ff=2048, seed=0):
    """Relative errors of the step's results against the fp32 layer."""
    args = inputs(rows, d, ff, seed)
    return {n: ((a.float() - b).norm() / b.norm()).item() for n, a, b in zip(NAMES, step(*args), plain_step(*args))}


if __name__ == "__main__":
    from dense_int8_matrix_gb300 import build
    build.build()
    for name, err in compare().items():
        print("%-8s relative error against fp32: %.5f" % (name, err))
