"""One training step of a layer of experts on the library's 8-bit operators.

    out = h + W2[e] silu(W1[e] norm(h)),   h = x + r,   e the row's expert

Forward: gemm_norm_f8 adds the residual, normalises and quantises; rows are
gathered by expert; two gemm_f8_grouped_run products with ragged rows, with
gemm_f8_quantize between them.  Backward: the products' input gradients (the
same grouped product with the transposed weights), the weights' gradients
(gemm_f8_quantize_cols and the product grouped along K) and
gemm_norm_backward.  gemm_balance counts the experts' rows; the router's
product, its argmax, the sort and the activation stay in torch.  `python examples/expert_layer.py` compares the step with
the same layer in fp32 torch.
"""

from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from dense_int8_matrix_gb300 import binding as B  # noqa: E402

F8 = torch.float8_e4m3fn
EPS = 1e-6


def f8_empty(*shape):
    """FP8 storage whose rows start at multiples of 16 bytes."""
    pitch = (shape[-1] + 15) // 16 * 16
    return torch.empty(*shape[:-1], pitch, dtype=F8, device="cuda")[..., :shape[-1]]


def quantise_weights(w):
    """FP8 copies of w (experts, n, k) in 128 x 128 blocks, for the forward
    product and, transposed, for the input gradient."""
    out = []
    for x in (w, w.transpose(1, 2).contiguous()):
        g, n, k = x.shape
        q, s = f8_empty(g, n, k), torch.empty(g, (n + 127) // 128, (k + 127) // 128, device="cuda")
        for i in range(g):   # blocks do not cross experts
            B.gemm_f8_quantize(x[i], q[i], s[i], B.GEMM_SCALE_BLOCKS)
        out.append((q, s))
    return out


def quantise_rows(x):
    q, s = f8_empty(*x.shape), torch.empty((x.shape[1] + 127) // 128, x.shape[0], device="cuda")
    B.gemm_f8_quantize(x, q, s)
    return q, s


def product(a, a_scale, weights, offsets):
    """Rows of a, grouped by offsets, times their experts' weights."""
    q, s = weights
    (m, k), (g, n, _) = a.shape, q.shape
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    B.gemm_f8_grouped_run(B.gemm_f8_grouped_plan(B.GEMM_GROUP_ROWS, g, m, k, n), a, a_scale, q, s, offsets, out)
    return out


def weight_gradient(dy, x, offsets):
    """dy^T x per expert, fp32."""
    m, g = dy.shape[0], offsets.shape[0] - 1
    kp = B.gemm_f8_padded_k(m, g)
    sides = []
    for t in (dy, x):
        q, s = f8_empty(t.shape[1], kp), torch.empty(kp // 128, t.shape[1], device="cuda")
        B.gemm_f8_quantize_cols(t, q, s, offsets)
        sides += [q, s]
    n, k = dy.shape[1], x.shape[1]
    dw = torch.empty(g, n, k, device="cuda")
    plan = B.gemm_f8_grouped_plan(B.GEMM_GROUP_K, g, n, kp, k, b_scale=B.GEMM_SCALE_ROWS)
    B.gemm_f8_grouped_run(plan, *sides, offsets, dw)
    return dw


def balance(logits, expert, coef=0.01):
    """Where the rows of each expert begin once they are sorted by it, and the
    loss that keeps the experts equally used."""
    rows, experts = logits.shape
    counts, offsets, used = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (experts, experts + 1, 1))
    lse, probs, loss = (torch.empty(n, device="cuda") for n in (rows, experts, 1))
    B.gemm_balance(logits, expert[:, None].to(torch.int32), coef, counts, offsets, used, lse, probs, loss)
    return offsets, loss


def step(x, r, norm_w, router, w1, w2, d_out):
    """Forward and backward.  x, r, d_out: (rows, d) bfloat16; norm_w: (d,)
    fp32; router: (experts, d); w1: (experts, ff, d), w2: (experts, d, ff)
    fp32.  Returns out, the gradient of x (and of r), and those of norm_w, w1
    and w2."""
    rows, d = x.shape
    experts = router.shape[0]
    (w1q, w1t), (w2q, w2t) = quantise_weights(w1), quantise_weights(w2)

    h, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    q, scale = f8_empty(rows, d), torch.empty((d + 127) // 128, rows, device="cuda")
    B.gemm_norm_f8(x, r, norm_w, EPS, h, rstd, q, scale)

    logits = h.float() @ router.T
    expert = logits.argmax(1)
    order = torch.argsort(expert, stable=True)
    offsets, _ = balance(logits, expert)

    a = f8_empty(rows, d)
    a.view(torch.uint8).copy_(q.view(torch.uint8)[order])
    a_scale = scale[:, order].contiguous()
    z = product(a, a_scale, w1q, offsets).float()
    gate = torch.sigmoid(z)
    hidden = (z * gate).to(torch.bfloat16)
    hq, hs = quantise_rows(hidden)
    y = product(hq, hs, w2q, offsets)
    out = h.clone().index_add_(0, order, y)

    dy = d_out[order].contiguous()
    dw2 = weight_gradient(dy, hidden, offsets)
    d_hidden = product(*quantise_rows(dy), w2t, offsets).float()
    d_z = (d_hidden * gate * (1 + z * (1 - gate))).to(torch.bfloat16)
    normed = (h.float() * rstd[:, None] * norm_w).to(torch.bfloat16)[order].contiguous()
    dw1 = weight_gradient(d_z, normed, offsets)
    d_norm = torch.empty_like(x)
    d_norm[order] = product(*quantise_rows(d_z), w1t, offsets)
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    B.gemm_norm_backward(d_norm, h, norm_w, rstd, d_out, dx, dw)
    return out, dx, dw, dw1, dw2


def plain_step(x, r, norm_w, router, w1, w2, d_out):
    """The same layer in fp32 torch with autograd; routed as the library's."""
    h0 = (x.float() + r.float()).to(torch.bfloat16).float()
    h, nw, a1, a2 = (t.detach().clone().requires_grad_(True) for t in (h0, norm_w, w1, w2))
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * nw
    expert = (h0 @ router.T).argmax(1)
    parts = torch.zeros_like(h)
    for e in range(router.shape[0]):
        rows = (expert == e).nonzero()[:, 0]
        parts = parts.index_add(0, rows, torch.nn.functional.silu(y[rows] @ a1[e].T) @ a2[e].T)
    out = h + parts
    out.backward(d_out.float())
    return out.detach(), h.grad, nw.grad, a1.grad, a2.grad


def inputs(rows, d, ff, experts, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (rand(rows, d).to(torch.bfloat16), rand(rows, d).to(torch.bfloat16), 1 + 0.1 * rand(d), rand(experts, d),
            rand(experts, ff, d) / d ** 0.5, rand(experts, d, ff) / ff ** 0.5, (0.1 * rand(rows, d)).to(torch.bfloat16))


def compare(rows=1000, d=512, ff=768, experts=6, seed=0):
    """Relative errors of the step's results against the fp32 layer."""
    args = inputs(rows, d, ff, experts, seed)
    names = ("out", "dx", "dnorm", "dw1", "dw2")
    return {n: ((a.float() - b).norm() / b.norm()).item()
            for n, a, b in zip(names, step(*args), plain_step(*args))}


if __name__ == "__main__":
    from dense_int8_matrix_gb300 import build
    build.build()
    for name, err in compare().items():
        print("%-6s relative error against fp32: %.4f" % (name, err))
