"""Measured cases of the bfloat16 layer's operators: the matrix product with
bias, activation and residual in its epilogue and the products of its backward
pass, the activation's gradient with the bias's, the layer norm and its
gradient, and the balance loss of a router with the experts' counts.

Each case runs either in plain torch operations in 32 bits (``own`` false) or
through the library's binding (``own`` true).  Shapes of products are (m, k, n)
as in the library: A is m x k, the weights are n x k, D is m x n.
"""

import math

import torch

own = False

EPS = 1e-5
COEF = 0.01
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a token of a decode step through a layer's first product: the weights' bytes
        {"name": "linear, one token", "op": "linear", "m": 1, "k": 8192, "n": 8192, "act": "silu", "residual": False, "keep": False},
        # a decode batch that fills no tile, onto the residual stream
        {"name": "linear, decode batch", "op": "linear", "m": 100, "k": 8192, "n": 8192, "act": "none", "residual": True, "keep": False},
        # odd sizes in every direction; rows of 777 elements start on any even byte
        {"name": "linear, ragged", "op": "linear", "m": 1000, "k": 777, "n": 3000, "act": "gelu", "residual": False, "keep": False},
        # the library's headline size, with what the backward pass needs kept
        {"name": "linear, 8192", "op": "linear", "m": 8192, "k": 8192, "n": 8192, "act": "gelu_tanh", "residual": False, "keep": True},
        # a layer's backward: input gradient through the activation before it, weight and bias gradients
        {"name": "linear backward", "op": "linear_back", "m": 4096, "k": 4096, "n": 4096, "act": "gelu"},
        # the same of a batch with no round size
        {"name": "linear backward, ragged", "op": "linear_back", "m": 2050, "k": 1206, "n": 777, "act": "silu"},
        # a wide layer's activation and bias in the backward pass: bandwidth
        {"name": "activation backward", "op": "act_back", "m": 4096, "n": 16384, "act": "gelu_tanh"},
        # a token of a decode step through one layer's norm: latency
        {"name": "layer norm, one token", "op": "norm", "rows": 1, "d": 8192, "x": "bf16", "y": "bf16"},
        # a long prompt's rows: bandwidth
        {"name": "layer norm, prompt", "op": "norm", "rows": 8192, "d": 8192, "x": "bf16", "y": "bf16"},
        # the norm's gradient in a training step
        {"name": "layer norm backward", "op": "norm_back", "rows": 4096, "d": 8192, "x": "bf16", "y": "bf16"},
        # a decode batch's router: counts and offsets for the experts' products, latency
        {"name": "balance, decode batch", "op": "balance", "rows": 48, "experts": 32, "top_k": 2, "x": "f32", "back": False},
        # a training batch over many experts, with the gradient of the loss
        {"name": "balance, training", "op": "balance", "rows": 65536, "experts": 256, "top_k": 8, "x": "f32", "back": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["linear", "linear", "linear", "linear_back", "linear_back", "act_back", "norm", "norm_back", "balance", "balance"])
    act = rng.choice(ACTS)
    if op == "linear":
        return {"op": op, "m": log(1, 8192), "k": log(64, 8192), "n": log(64, 8192), "act": act,
                "residual": rng.random() < 0.4, "keep": rng.random() < 0.4}
    if op == "linear_back":
        return {"op": op, "m": log(64, 4096), "k": log(64, 4096), "n": log(64, 4096), "act": act}
    if op == "act_back":
        n = log(64, 16384)
        return {"op": op, "m": log(1, (4096 * 16384) // n), "n": n, "act": act}
    if op in ("norm", "norm_back"):
        d = log(64, 16384)
        return {"op": op, "rows": log(1, (4096 * 8192) // d), "d": d, "x": rng.choice(["bf16", "f32"]),
                "y": rng.choice(["bf16", "bf16", "f32"])}
    experts = log(4, 512)
    return {"op": op, "rows": log(1, (65536 * 256) // experts), "experts": experts,
            "top_k": min(experts, rng.choice([1, 2, 4, 8])), "x": rng.choice(["bf16", "f32"]), "back": rng.random() < 0.6}


# ---------------------------------------------------------------- the inputs --

def activations(rows, d, g):
    """N(0, 1) with a spread of scales over the channels and a few outlier ones."""
    spread = torch.exp(0.4 * torch.randn(d, generator=g, device="cuda"))
    spread[torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")] *= 12.0
    return torch.randn(rows, d, generator=g, device="cuda") * spread


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    bf16, f32, dev = torch.bfloat16, torch.float32, {"device": "cuda"}

    def randn(*shape):
        return torch.randn(*shape, generator=g, **dev)

    if op in ("linear", "linear_back"):
        m, k, n = case["m"], case["k"], case["n"]
        w = (randn(n, k) / k ** 0.5).to(bf16)
        if op == "linear":
            s["a"], s["w"], s["bias"] = activations(m, k, g).to(bf16), w, 0.1 * randn(n)
            s["r"] = activations(m, n, g).to(bf16) if case["residual"] else None
            s["z"] = torch.empty(m, n, dtype=bf16, **dev) if case["keep"] else None
            s["out"] = torch.empty(m, n, dtype=bf16, **dev)
        else:
            # dz: the gradient of this layer's sums; zp: the sums of the layer
            # before, whose activation made x
            s["dz"], s["x"], s["w"], s["zp"] = (0.02 * randn(m, n)).to(bf16), activations(m, k, g).to(bf16), w, randn(m, k).to(bf16)
            s["dzp"] = torch.empty(m, k, dtype=bf16, **dev)
            s["dw"], s["db"] = torch.empty(n, k, dtype=f32, **dev), torch.empty(n, dtype=f32, **dev)
    elif op == "act_back":
        m, n = case["m"], case["n"]
        s["dy"], s["z"] = (0.02 * randn(m, n)).to(bf16), randn(m, n).to(bf16)
        s["dz"], s["db"] = torch.empty(m, n, dtype=bf16, **dev), torch.empty(n, dtype=f32, **dev)
    elif op in ("norm", "norm_back"):
        rows, d, tx, ty = case["rows"], case["d"], TYPES[case["x"]], TYPES[case["y"]]
        s["w"], s["b"] = 1.0 + 0.1 * randn(d), 0.1 * randn(d)
        x, r = (activations(rows, d, g) + 0.3).to(tx), activations(rows, d, g).to(tx)
        if op == "norm":
            s["x"], s["r"], s["h"], s["out"] = x, r, torch.empty_like(x), torch.empty(rows, d, dtype=ty, **dev)
            s["mean"], s["rstd"] = torch.empty(rows, **dev), torch.empty(rows, **dev)
        else:
            h = x.float()
            s["h"], s["dr"] = x, (0.02 * r.float()).to(tx)   # dr: the gradient that reaches h as the residual
            s["mean"] = h.mean(-1)
            s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(-1) + EPS)
            s["dy"] = (0.02 * randn(rows, d)).to(ty)
            s["dx"], s["dw"], s["db"] = torch.empty_like(x), torch.empty(d, **dev), torch.empty(d, **dev)
    else:
        rows, e, k = case["rows"], case["experts"], case["top_k"]
        # popularity of the experts and the rows' own tastes
        s["x"] = (randn(rows, e) + 0.7 * randn(e)).to(TYPES[case["x"]])
        index = s["x"].float().topk(k, dim=1).indices.to(torch.int32)
        # a padded batch: no row has an expert behind the last token; and a
        # few slots that a full expert has turned away
        index[torch.rand(rows, k, generator=g, **dev) < 0.02] = -1
        index[rows - rows // 16:] = -1
        s["index"] = index.contiguous()
        s["counts"], s["offsets"] = torch.empty(e, dtype=torch.int32, **dev), torch.empty(e + 1, dtype=torch.int32, **dev)
        s["used"], s["lse"] = torch.empty(1, dtype=torch.int32, **dev), torch.empty(rows, **dev)
        s["probs"], s["loss"] = torch.empty(e, **dev), torch.empty(1, **dev)
        if case["back"]:
            s["dloss"] = torch.full((1,), 0.5, **dev)
            s["dr"] = (0.001 * randn(rows, e)).to(s["x"].dtype)   # the gradient through the gates
            s["dx"] = torch.empty_like(s["x"])
    if own:
        # the plans that a program makes once for a shape and keeps
        from dense_int8_matrix_gb300 import binding as B
        s["act_code"] = getattr(B, "GEMM_ACT_" + case.get("act", "none").upper())
        if op == "linear":
            s["plan"] = B.gemm_bf16_linear_plan(m, k, n)
        elif op == "linear_back":
            s["plan"] = B.gemm_bf16_linear_plan(m, n, k, B.GEMM_FORM_NN)
            s["plan_w"] = B.gemm_bf16_linear_plan(n, m, k, B.GEMM_FORM_TN)
    return s


# ----------------------------------------------------------- the plain forms --

def act_of(name, v):
    if name == "relu":
        return torch.where(v > 0, v, 0.0)
    if name == "gelu":
        return v * 0.5 * torch.erfc(v * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-2.0 * c * (z + 0.044715 * z * z * z)))
        return s + 2.0 * z * s * (1.0 - s) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def plain_balance(s):
    e, x, index = s["experts"], s["x"].float(), s["index"].long()
    taken = (index >= 0) & (index < e)
    used = taken.any(1)
    counts = torch.zeros(e + 1, dtype=torch.int32, device=x.device)
    counts.scatter_add_(0, torch.where(taken, index, e).flatten(), torch.ones_like(index, dtype=torch.int32).flatten())
    counts = counts[:e]
    top = x.amax(1, keepdim=True)
    ex = torch.exp(x - top)
    total = ex.sum(1, keepdim=True)
    p = torch.where(used[:, None], ex / total, 0.0)
    rows = used.sum().clamp_min(1)
    probs = p.sum(0) / rows
    share = counts / counts.sum().clamp_min(1)
    out = {"counts": counts, "offsets": torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32),
           "used": used.sum().to(torch.int32).reshape(1),
           "lse": torch.where(used, (top + torch.log(total))[:, 0], math.inf), "probs": probs,
           "loss": (COEF * e * (share * probs).sum()).reshape(1)}
    if s["back"]:
        scale = s["dloss"] * COEF * e / rows
        d = scale * p * (share - (p * share).sum(1, keepdim=True))
        out["dx"] = (s["dr"].float() + d).to(s["dr"].dtype)
    return out


def plain(s):
    op, act = s["op"], s.get("act")
    if op == "linear":
        v = s["a"].float() @ s["w"].float().T + s["bias"]
        y = act_of(act, v)
        if s["r"] is not None:
            y = y + s["r"].float()
        out = {"out": y.to(torch.bfloat16)}
        if s["keep"]:
            out["z"] = v.to(torch.bfloat16)
        return out
    if op == "linear_back":
        dz = s["dz"].float()
        dzp = (dz @ s["w"].float()) * act_slope(act, s["zp"].float())
        return {"dzp": dzp.to(torch.bfloat16), "dw": dz.T @ s["x"].float(), "db": dz.sum(0)}
    if op == "act_back":
        dz = s["dy"].float() * act_slope(act, s["z"].float())
        return {"dz": dz.to(torch.bfloat16), "db": dz.sum(0)}
    if op == "norm":
        h = (s["x"].float() + s["r"].float()).to(s["x"].dtype)
        hf = h.float()
        mean = hf.mean(-1)
        c = hf - mean[:, None]
        rstd = torch.rsqrt(c.square().mean(-1) + EPS)
        return {"h": h, "mean": mean, "rstd": rstd, "out": (c * rstd[:, None] * s["w"] + s["b"]).to(TYPES[s["y"]])}
    if op == "norm_back":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["h"].float() - s["mean"][:, None]) * rstd
        gy = dy * s["w"]
        dx = s["dr"].float() + rstd * (gy - gy.mean(-1, keepdim=True) - xhat * (gy * xhat).mean(-1, keepdim=True))
        return {"dx": dx.to(s["h"].dtype), "dw": (dy * xhat).sum(0), "db": dy.sum(0)}
    return plain_balance(s)


# ------------------------------------------------------- the library's calls --

def library(s):
    from dense_int8_matrix_gb300 import binding as B
    op, act = s["op"], s["act_code"]
    if op == "linear":
        B.gemm_bf16_linear_run(s["plan"], s["a"], s["w"], s["out"], bias=s["bias"], activation=act, Z=s["z"], residual=s["r"])
        return {"out": s["out"], "z": s["z"]} if s["keep"] else {"out": s["out"]}
    if op == "linear_back":
        B.gemm_bf16_linear_run(s["plan"], s["dz"], s["w"], s["dzp"], activation=act | B.GEMM_ACT_GRADIENT, Z=s["zp"])
        B.gemm_bf16_linear_run(s["plan_w"], s["dz"], s["x"], s["dw"])
        B.gemm_activation_backward(s["dz"], None, B.GEMM_ACT_NONE, None, s["db"])
        return {"dzp": s["dzp"], "dw": s["dw"], "db": s["db"]}
    if op == "act_back":
        B.gemm_activation_backward(s["dy"], s["z"], act, s["dz"], s["db"])
        return {"dz": s["dz"], "db": s["db"]}
    if op == "norm":
        B.gemm_layer_norm(s["x"], s["r"], s["w"], s["b"], EPS, s["h"], s["mean"], s["rstd"], s["out"])
        return {"h": s["h"], "mean": s["mean"], "rstd": s["rstd"], "out": s["out"]}
    if op == "norm_back":
        B.gemm_layer_norm_backward(s["dy"], s["h"], s["w"], s["mean"], s["rstd"], s["dr"], s["dx"], s["dw"], s["db"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    B.gemm_balance(s["x"], s["index"], COEF, s["counts"], s["offsets"], s["used"], s["lse"], s["probs"], s["loss"])
    names = ["counts", "offsets", "used", "lse", "probs", "loss"]
    if s["back"]:
        B.gemm_balance_backward(s["x"], s["lse"], s["counts"], s["used"], COEF, s["dloss"], s["dr"], s["dx"])
        names.append("dx")
    return {name: s[name] for name in names}


def run(state):
    return library(state) if own else plain(state)


# ---------------------------------------------------------- work, and truth --

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("linear", "linear_back"):
        m, k, n = case["m"], case["k"], case["n"]
        if op == "linear":   # A, the weights and D at 2 bytes, the residual, the kept sums, the bias
            return {"bytes": 2 * (m * k + n * k + m * n * (1 + case["residual"] + case["keep"])) + 4 * n, "flops": 2 * m * k * n}
        # dz, x, the weights, the sums before and their gradient at 2 bytes, dW and db at 4
        return {"bytes": 2 * (m * n + 3 * m * k + n * k) + 4 * (n * k + n), "flops": 4 * m * k * n + m * n}
    if op == "act_back":
        mn = case["m"] * case["n"]
        return {"bytes": 2 * mn * (3 if case["act"] != "none" else 2) + 4 * case["n"], "flops": 10 * mn}
    if op in ("norm", "norm_back"):
        rows, d, x, y = case["rows"], case["d"], size[case["x"]], size[case["y"]]
        if op == "norm":   # x, r, h and y; the statistics; w and b
            return {"bytes": rows * d * (3 * x + y) + 8 * rows + 8 * d, "flops": 10 * rows * d}
        return {"bytes": rows * d * (3 * x + y) + 8 * rows + 12 * d, "flops": 16 * rows * d}   # h, dr, dx and dy
    rows, e, x = case["rows"], case["experts"], size[case["x"]]
    index = 4 * rows * case["top_k"] + 4 * rows + 12 * e
    if case["back"]:   # the logits, the gradient's two sides; read once if both passes shared them
        return {"bytes": 3 * rows * e * x + index, "flops": 14 * rows * e}
    return {"bytes": rows * e * x + index, "flops": 6 * rows * e}


def truth_act(name, v):
    """The activation and its slope in 64 bits."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "relu":
        return v.clamp(min=0.0), torch.where(v > 0.0, 1.0, 0.0).double()
    if name == "silu":
        s = torch.reciprocal(1.0 + torch.exp(-v))
        return v * s, s + v * s * torch.reciprocal(1.0 + torch.exp(v))
    if name == "gelu":
        cdf = torch.erfc(-v / 2.0 ** 0.5) / 2.0
        return v * cdf, cdf + v * torch.exp(-v.square() / 2.0) / (2.0 * math.pi) ** 0.5
    u = (2.0 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3)
    low = torch.reciprocal(1.0 + torch.exp(-2.0 * u))    # (1 + tanh u) / 2
    high = torch.reciprocal(1.0 + torch.exp(2.0 * u))    # (1 - tanh u) / 2
    return v * low, low + 2.0 * v * low * high * (2.0 / math.pi) ** 0.5 * (1.0 + 0.134145 * v.square())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        v = torch.einsum("ik,jk->ij", s["a"].double(), s["w"].double()).add_(s["bias"].double())
        y = truth_act(case["act"], v)[0]
        if case["residual"]:
            y = y + s["r"].double()
        return {"out": y, "z": v} if case["keep"] else {"out": y}
    if op == "linear_back":
        dz = s["dz"].double()
        slope = truth_act(case["act"], s["zp"].double())[1]
        return {"dzp": torch.einsum("ij,jk->ik", dz, s["w"].double()) * slope,
                "dw": torch.einsum("ij,ik->jk", dz, s["x"].double()), "db": torch.einsum("ij->j", dz)}
    if op == "act_back":
        dz = truth_act(case["act"], s["z"].double())[1].mul_(s["dy"].double())
        return {"dz": dz, "db": torch.einsum("ij->j", dz)}
    if op == "norm":
        h = (s["x"].double() + s["r"].double()).to(s["x"].dtype).double()
        var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
        rstd = 1.0 / torch.sqrt(var + EPS)
        return {"h": h, "mean": mean[:, 0], "rstd": rstd[:, 0], "out": (h - mean) * rstd * s["w"].double() + s["b"].double()}
    if op == "norm_back":
        h, dy, w, d = s["h"].double(), s["dy"].double(), s["w"].double(), case["d"]
        r = s["rstd"].double()
        c = h - s["mean"].double()[:, None]
        dot = torch.einsum("ij,ij,j->i", dy, c, w) / d
        dx = s["dr"].double() + (dy * w - (torch.einsum("ij,j->i", dy, w) / d)[:, None]) * r[:, None] - c * (r ** 3 * dot)[:, None]
        return {"dx": dx, "dw": torch.einsum("ij,ij,i->j", dy, c, r), "db": torch.einsum("ij->j", dy)}
    e, rows = case["experts"], case["rows"]
    index = s["index"]
    valid = torch.stack([(index == i).sum() for i in range(e)])
    used = (index >= 0).sum(1) > 0
    x = s["x"].double()
    lse = torch.where(used, torch.logsumexp(x, 1), math.inf)
    p = torch.where(used[:, None], torch.exp(x - torch.where(used, lse, 0.0)[:, None]), 0.0)
    t = max(int(used.sum()), 1)
    share = valid.double() / max(int(valid.sum()), 1)
    ends = torch.tensor([0] + valid.cumsum(0).tolist(), device=x.device)
    out = {"counts": valid, "offsets": ends, "used": used.sum().reshape(1), "lse": lse, "probs": torch.einsum("ij->j", p) / t,
           "loss": (COEF * e / t * torch.einsum("ij,j->", p, share)).reshape(1)}
    if case["back"]:
        mix = torch.einsum("ij,j->i", p, share)
        out["dx"] = s["dr"].double() + s["dloss"].double() * COEF * e / t * (p * share - p * mix[:, None])
    return out
