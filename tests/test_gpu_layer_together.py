"""The bfloat16 layer's operators one after the other, as a model calls them.

Tolerances.  A rounding to bfloat16 is off by 2^-8 of the value at most, by
2^-8 / sqrt(3) = 0.23 % rms at worst.  The longest chains (the first weights'
gradient, the input's) pass through five such roundings, 0.5 %; z's rounding
also moves the activation's slope, by up to 0.8 |z| of it where the slope is
about one, so that up to four times that is allowed: 2 %.  A forgotten term or a
wrong row is tens of percent."""

import os
import sys

import pytest
import torch

from dense_int8_matrix_gb300 import binding as B

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_int8_matrix_gb300 import build
    build.build()
    yield
    st, code = B.gemm_device_error()
    assert st == B.GEMM_OK, "device error word set: code %d" % code


def error(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


@pytest.mark.parametrize("rows,d,ff", [(1000, 512, 2048), (129, 250, 1000), (70, 99, 333), (1, 64, 100), (2100, 128, 130)])
def test_dense_layer_step(rows, d, ff):
    import dense_layer
    args = dense_layer.inputs(rows, d, ff, seed=rows)
    got, want = dense_layer.step(*args), dense_layer.plain_step(*args, dtype=torch.float64)
    errors = {n: error(a, b) for n, a, b in zip(dense_layer.NAMES, got, want)}
    assert all(e < 0.02 for e in errors.values()), errors


def test_dense_layer_step_against_differences():
    import dense_layer
    args = list(dense_layer.inputs(12, 40, 72, seed=5))
    got = dict(zip(dense_layer.NAMES, dense_layer.step(*args)))

    def loss(a):   # the 64-bit layer; x + r is not rounded, so that it has differences
        x, r, nw, nb, w1, b1, w2, b2, g = a
        h = x + r
        y = torch.nn.functional.layer_norm(h, h.shape[1:], nw, nb, dense_layer.EPS)
        return ((h + torch.nn.functional.gelu(y @ w1.T + b1) @ w2.T + b2) * g).sum()

    exact = [a.double() for a in args]
    exact[0] = (args[0].double() + args[1].double()).to(torch.bfloat16).double()
    exact[1] = torch.zeros_like(exact[0])
    step = 1e-5
    for i, name in ((0, "dx"), (2, "dnorm_w"), (3, "dnorm_b"), (4, "dw1"), (5, "db1"), (6, "dw2"), (7, "db2")):
        # along a fixed random direction: one number that every element takes part in
        g = torch.Generator(device="cuda")
        g.manual_seed(i)
        way = torch.randn(exact[i].shape, generator=g, device="cuda", dtype=torch.float64)
        two = [loss(exact[:i] + [exact[i] + s * way] + exact[i + 1:]).item() for s in (step, -step)]
        slope = (two[0] - two[1]) / (2 * step)
        along = (got[name].double() * way).sum().item()
        assert abs(along - slope) <= 0.02 * got[name].double().norm().item() * way.norm().item() / got[name].numel() ** 0.5 * 3, name


@pytest.mark.parametrize("rows,d,ff", [(333, 136, 520), (700, 99, 333)])
def test_dense_layer_step_captured(rows, d, ff):
    import dense_layer
    first, second = dense_layer.inputs(rows, d, ff, seed=1), dense_layer.inputs(rows, d, ff, seed=2)
    want = [dense_layer.step(*a) for a in (first, second)]
    graphs = []
    for _ in range(2):   # two graphs of the same step, replayed on two streams at once
        args = [t.clone() for t in first]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = dense_layer.step(*args)
        graphs.append((graph, args, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for source, expect in ((second, want[1]), (first, want[0])):
        for _, args, _ in graphs:
            for t, s in zip(args, source):
                t.copy_(s)
        torch.cuda.synchronize()
        for _ in range(3):
            for (graph, _, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        eager = dense_layer.step(*source)   # beside them
        torch.cuda.synchronize()
        for _, _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, expect))
        assert all(torch.equal(a, b) for a, b in zip(eager, expect))


@pytest.mark.parametrize("rows,d,ff,experts,top_k", [(500, 256, 384, 8, 2), (3, 128, 128, 5, 1), (1000, 200, 136, 33, 4)])
def test_routed_layer(rows, d, ff, experts, top_k):
    """Layer norm, the router's product, the balance loss with the offsets that
    the grouped FP8 product takes, and the way back to the layer's input."""
    import dense_layer
    import expert_layer
    product, coef, F64 = dense_layer.product, 0.01, torch.float64
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf16 = torch.bfloat16
    x, r, d_h = rand(rows, d).to(bf16), rand(rows, d).to(bf16), (0.001 * rand(rows, d)).to(bf16)
    nw, nb, router, w = 1 + 0.1 * rand(d), 0.1 * rand(d), (rand(experts, d) / d ** 0.5).to(bf16), rand(experts, ff, d) / d ** 0.5

    h, y = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    B.gemm_layer_norm(x, r, nw, nb, 1e-5, h, mean, rstd, y)
    logits = product(B.GEMM_FORM_NT, y, router)
    index = logits.float().topk(top_k, 1).indices.to(torch.int32)
    counts, offsets, used = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (experts, experts + 1, 1))
    lse, probs, loss = (torch.empty(n, device="cuda") for n in (rows, experts, 1))
    B.gemm_balance(logits, index, coef, counts, offsets, used, lse, probs, loss)
    order = torch.argsort(index.flatten(), stable=True)
    q, s = expert_layer.quantise_rows(y[order // top_k].contiguous())
    z = expert_layer.product(q, s, expert_layer.quantise_weights(w)[0], offsets)
    want_z = torch.einsum("md,mfd->mf", y[order // top_k].double(), w.to(F64)[index.flatten()[order].long()])
    # (three fraction bits for both factors: 5.1 % rms at worst)
    assert error(z, want_z) < 0.1

    d_loss = torch.ones(1, device="cuda")
    d_logits = torch.empty_like(logits)
    B.gemm_balance_backward(logits, lse, counts, used, coef, d_loss, None, d_logits)
    d_router = product(B.GEMM_FORM_TN, d_logits, y, torch.float32)
    d_y = product(B.GEMM_FORM_NN, d_logits, router)
    dx, dnw, dnb = torch.empty_like(x), torch.empty_like(nw), torch.empty_like(nb)
    B.gemm_layer_norm_backward(d_y, h, nw, mean, rstd, d_h, dx, dnw, dnb)

    leaves = [t.to(F64).requires_grad_(True) for t in (h, nw, nb, router)]
    y64 = torch.nn.functional.layer_norm(leaves[0], (d,), leaves[1], leaves[2], 1e-5)
    p = (y64 @ leaves[3].T).softmax(1)
    f = torch.bincount(index.flatten().long(), minlength=experts).to(F64) / index.numel()
    want = coef * experts * (f * p.mean(0)).sum()
    grads = torch.autograd.grad(want + (leaves[0] * d_h.to(F64)).sum(), leaves)
    assert abs(loss.item() / want.item() - 1) < 0.02
    assert torch.equal(counts.cpu().long(), torch.bincount(index.flatten().long().cpu(), minlength=experts))
    for got, wanted in zip((dx, dnw, dnb, d_router), grads):
        assert error(got, wanted) < 0.02
