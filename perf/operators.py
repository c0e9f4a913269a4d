"""Measured cases of the 8-bit operators: the RMS norm with the residual's
addition (8-bit output with scales, and its gradient), the FP8 matrix product
with a scale for each block of 128, the same product grouped by expert, and the
FP8 quantisation that feeds the backward products.

Each case runs either in plain torch operations in 32 bits (``own`` false) or
through the library's binding (``own`` true).  Shapes are (m, k, n) as in the
library: A is m x k, Bt is n x k, D is m x n.  Scales of 1 x 128 blocks are
stored block-major, (ceil(k / 128), rows); scales of 128 x 128 blocks are
(ceil(n / 128), ceil(k / 128)).
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
BLOCK = 128
TINY = 2.0 ** -126
EPS = 1e-6


def listed():
    return [
        # a token of a decode step through one layer's norm: latency
        {"name": "norm f8, one token", "op": "norm_f8", "rows": 1, "d": 8192},
        # a long prompt's rows through the same norm: bandwidth
        {"name": "norm f8, prompt", "op": "norm_f8", "rows": 8192, "d": 8192},
        # an odd width, a row scale, and the int8 product that reads it
        {"name": "norm i8 and int8 product", "op": "norm_i8", "rows": 1000, "d": 777, "n": 3000},
        # the norm's gradient in a training step
        {"name": "norm backward", "op": "norm_back", "rows": 4096, "d": 8192},
        # one token against a layer's weights: the weights' bytes
        {"name": "product, one token", "op": "gemm", "m": 1, "k": 8192, "n": 8192},
        # a decode batch of a size that fills no tile
        {"name": "product, decode batch", "op": "gemm", "m": 100, "k": 8192, "n": 8192},
        # odd sizes in every direction
        {"name": "product, ragged", "op": "gemm", "m": 1000, "k": 777, "n": 3000},
        # the library's headline size
        {"name": "product, 8192", "op": "gemm", "m": 8192, "k": 8192, "n": 8192},
        # a linear layer's backward: quantise dY both ways and X, dX and dW
        {"name": "linear backward", "op": "gemm_back", "m": 4096, "k": 4096, "n": 4096},
        # a decode batch spread over experts, most with one or two rows, some with none
        {"name": "experts, decode batch", "op": "grouped", "m": 48, "k": 4096, "n": 4096, "groups": 32, "skew": 1.0},
        # a prompt over the same experts, unevenly
        {"name": "experts, prompt", "op": "grouped", "m": 8200, "k": 4096, "n": 2048, "groups": 32, "skew": 1.0},
        # the experts' backward: dX by rows and dW by tokens of each expert
        {"name": "experts backward", "op": "grouped_back", "m": 4099, "k": 2048, "n": 1024, "groups": 8, "skew": 1.0},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm_f8", "norm_i8", "norm_back", "gemm", "gemm", "gemm_back", "grouped", "grouped", "grouped_back"])
    if op in ("norm_f8", "norm_back"):
        d = log(256, 16384)
        return {"op": op, "rows": log(1, (8192 * 8192) // d), "d": d}
    if op == "norm_i8":
        return {"op": op, "rows": log(1, 4096), "d": log(256, 4096), "n": log(256, 4096)}
    if op == "gemm":
        return {"op": op, "m": log(1, 8192), "k": log(256, 8192), "n": log(256, 8192)}
    if op == "gemm_back":
        return {"op": op, "m": log(64, 4096), "k": log(256, 4096), "n": log(256, 4096)}
    groups = log(2, 64)
    skew = rng.choice([0.0, 0.5, 1.0])
    if op == "grouped":
        return {"op": op, "m": log(4, 8200), "k": log(256, 4096), "n": log(256, 4096), "groups": groups, "skew": skew}
    return {"op": op, "m": log(64, 4099), "k": log(256, 2048), "n": log(256, 2048), "groups": min(groups, 16), "skew": skew}


# ---------------------------------------------------------------- the inputs --

def blocks_of(k):
    return (k + BLOCK - 1) // BLOCK


def pitch_of(k):
    return (k + 15) // 16 * 16


def activations(rows, d, g):
    """N(0, 1) with a spread of scales over the channels and a few outlier ones, as bfloat16."""
    spread = torch.exp(0.4 * torch.randn(d, generator=g, device="cuda"))
    spread[torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")] *= 12.0
    return (torch.randn(rows, d, generator=g, device="cuda") * spread).to(torch.bfloat16)


def f8_matrix(rows, k):
    """rows x k, row pitch a multiple of 16 bytes."""
    return torch.zeros(rows, pitch_of(k), dtype=F8, device="cuda")[:, :k]


def blocked(x):
    """(rows, k) as (rows, blocks, 128), padded with zeros."""
    kb = blocks_of(x.shape[-1])
    return torch.nn.functional.pad(x, (0, kb * BLOCK - x.shape[-1])).unflatten(-1, (kb, BLOCK))


def quantised_rows(x):
    """e4m3 values and scales (blocks, rows) of x (rows, k) in 1 x 128 blocks."""
    xb = blocked(x)
    scale = (xb.abs().amax(-1) / F8_MAX).clamp_min(TINY)
    q = (xb * (1.0 / scale).unsqueeze(-1)).flatten(-2)[..., : x.shape[-1]].to(F8)
    return q, scale.transpose(-1, -2)


def quantised_blocks(x):
    """e4m3 values and scales (row blocks, blocks) of x (..., rows, k) in 128 x 128 blocks."""
    rows, k = x.shape[-2:]
    rb, kb = blocks_of(rows), blocks_of(k)
    xp = torch.nn.functional.pad(x, (0, kb * BLOCK - k, 0, rb * BLOCK - rows))
    xp = xp.unflatten(-1, (kb, BLOCK)).unflatten(-3, (rb, BLOCK))
    scale = (xp.abs().amax((-3, -1)) / F8_MAX).clamp_min(TINY)
    q = (xp * (1.0 / scale)[..., :, None, :, None]).flatten(-4, -3).flatten(-2)[..., :rows, :k]
    return q.to(F8), scale


def expert_sizes(case, g):
    """Rows of each expert: popularity falls with `skew`, some experts get none."""
    w = torch.arange(1, case["groups"] + 1, device="cuda", dtype=torch.float32).pow(-case["skew"])
    w = w[torch.randperm(case["groups"], generator=g, device="cuda")]
    pick = torch.multinomial(w, case["m"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=case["groups"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    dev = {"device": "cuda"}
    if op in ("norm_f8", "norm_i8", "norm_back"):
        rows, d = case["rows"], case["d"]
        s["h"] = torch.empty(rows, d, dtype=torch.bfloat16, **dev)
        s["rstd"] = torch.empty(rows, **dev)
        s["w"] = 1.0 + 0.1 * torch.randn(d, generator=g, **dev)
        s["x"], s["r"] = activations(rows, d, g), activations(rows, d, g)
        if op == "norm_f8":
            s["q"], s["scale"] = f8_matrix(rows, d), torch.empty(blocks_of(d), rows, **dev)
        elif op == "norm_i8":
            s["q"], s["scale"] = torch.empty(rows, d, dtype=torch.int8, **dev), torch.empty(rows, **dev)
            s["wt"] = (32 * torch.randn(case["n"], d, generator=g, **dev)).round().clamp(-127, 127).to(torch.int8)
            s["col_scale"] = (0.5 + torch.rand(case["n"], generator=g, **dev)) / 1600
            s["out"] = torch.empty(rows, case["n"], dtype=torch.bfloat16, **dev)
        else:
            h = s["h"] = s.pop("x")
            s["dr"] = (0.02 * s.pop("r").float()).to(torch.bfloat16)   # the gradient of h as the residual
            s["dy"] = (0.02 * torch.randn(rows, d, generator=g, **dev)).to(torch.bfloat16)
            s["rstd"] = torch.rsqrt(h.float().square().mean(-1) + EPS)
            s["dx"], s["dw"] = torch.empty_like(h), torch.empty(d, **dev)
    else:
        m, k, n = case["m"], case["k"], case["n"]
        groups = case.get("groups", 0)
        if groups:
            sizes = expert_sizes(case, g)
            s["offsets"] = torch.nn.functional.pad(sizes.cumsum(0), (1, 0)).to(torch.int32)
            s["most"] = int(sizes.max())
        w = 0.02 * torch.randn(max(groups, 1), n, k, generator=g, **dev)
        x = activations(m, k, g)
        if op in ("gemm", "grouped"):
            a, s["a_scale"] = quantised_rows(x.float())
            s["a"] = f8_matrix(m, k)
            s["a"].copy_(a)
            s["a_scale"] = s["a_scale"].contiguous()
            s["out"] = torch.empty(m, n, dtype=torch.bfloat16, **dev)
        else:
            w = w.transpose(1, 2).contiguous()   # dX = dY W: the weights' columns are the contraction
            s["x"] = x
            s["dy"] = (0.02 * torch.randn(m, n, generator=g, **dev)).to(torch.bfloat16)
            kp = (m + 127 * max(groups, 1)) // BLOCK * BLOCK
            s["dy_q"], s["dy_s"] = f8_matrix(m, n), torch.empty(blocks_of(n), m, **dev)
            s["dy_qc"], s["dy_sc"] = torch.empty(n, kp, dtype=F8, **dev), torch.empty(kp // BLOCK, n, **dev)
            s["x_qc"], s["x_sc"] = torch.empty(k, kp, dtype=F8, **dev), torch.empty(kp // BLOCK, k, **dev)
            s["dx"] = torch.empty(m, k, dtype=torch.bfloat16, **dev)
            s["dw"] = torch.empty(max(groups, 1), n, k, **dev) if groups else torch.empty(n, k, **dev)
        rows_b, k_b = w.shape[1:]
        b, b_scale = quantised_blocks(w)
        bt = torch.zeros(max(groups, 1), rows_b, pitch_of(k_b), dtype=F8, **dev)[:, :, :k_b]
        bt.copy_(b)
        s["b"], s["b_scale"] = (bt, b_scale.contiguous()) if groups else (bt[0], b_scale[0].contiguous())
    if own:
        # the plans that a program makes once for a shape and keeps
        from dense_int8_matrix_gb300 import binding as B
        if op == "norm_i8":
            s["plan"] = B.gemm_i8_plan(case["rows"], case["d"], case["n"])
        elif op == "gemm":
            s["plan"] = B.gemm_f8_plan(m, k, n)
        elif op == "grouped":
            s["plan"] = B.gemm_f8_grouped_plan(B.GEMM_GROUP_ROWS, groups, m, k, n)
        elif op == "gemm_back":
            s["plan"] = B.gemm_f8_plan(m, n, k)
            s["plan_w"] = B.gemm_f8_plan(n, kp, k, b_scale=B.GEMM_SCALE_ROWS)
        elif op == "grouped_back":
            s["plan"] = B.gemm_f8_grouped_plan(B.GEMM_GROUP_ROWS, groups, m, n, k)
            s["plan_w"] = B.gemm_f8_grouped_plan(B.GEMM_GROUP_K, groups, n, kp, k, b_scale=B.GEMM_SCALE_ROWS)
    return s


# ----------------------------------------------------------- the plain forms --

def plain_norm(s):
    h = (s["x"].float() + s["r"].float()).to(torch.bfloat16)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(-1) + EPS)
    return h, rstd, hf * rstd.unsqueeze(-1) * s["w"]


def scaled_rows(q, scale):
    """The values that 1 x 128 blocks stand for: q (rows, k), scale (blocks, rows)."""
    return (blocked(q.float()) * scale.transpose(-1, -2).unsqueeze(-1)).flatten(-2)[..., : q.shape[-1]]


def scaled_blocks(q, scale):
    """The values that 128 x 128 blocks stand for: q (..., n, k), scale (..., row blocks, blocks)."""
    n, k = q.shape[-2:]
    full = scale.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]
    return q.float() * full


def padded_groups(s, x):
    """x's rows by group, (groups, most, columns), zeros behind each group's rows; and the index of each row there."""
    off = s["offsets"].long()
    step = torch.arange(s["most"], device=x.device)
    at = off[:-1, None] + step
    inside = at < off[1:, None]
    rows = torch.arange(x.shape[0], device=x.device)
    group = torch.searchsorted(off, rows, right=True) - 1
    return torch.where(inside.unsqueeze(-1), x[at.clamp_max(x.shape[0] - 1)], 0.0), group, rows - off[group]


def plain_weight_gradient(dy, x):
    """dY^T X over the rows (tokens), both quantised in blocks of 128 tokens."""
    dq, ds = quantised_rows(dy.transpose(-1, -2))
    xq, xs = quantised_rows(x.transpose(-1, -2))
    return scaled_rows(dq, ds) @ scaled_rows(xq, xs).transpose(-1, -2)


def plain(s):
    op = s["op"]
    if op == "norm_f8":
        h, rstd, y = plain_norm(s)
        q, scale = quantised_rows(y)
        return {"h": h, "rstd": rstd, "q": q, "scale": scale}
    if op == "norm_i8":
        h, rstd, y = plain_norm(s)
        scale = (y.abs().amax(-1) / 127.0).clamp_min(TINY)
        q = (y * (1.0 / scale).unsqueeze(-1)).round().clamp(-127, 127)
        out = (q @ s["wt"].float().T) * scale.unsqueeze(-1) * s["col_scale"]
        return {"h": h, "rstd": rstd, "scale": scale, "out": out.to(torch.bfloat16)}
    if op == "norm_back":
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(-1)
        xhat = s["h"].float() * rstd
        gy = dy * s["w"]
        dx = s["dr"].float() + rstd * (gy - xhat * (gy * xhat).mean(-1, keepdim=True))
        return {"dx": dx.to(torch.bfloat16), "dw": (dy * xhat).sum(0)}
    if op == "gemm":
        return {"out": (scaled_rows(s["a"], s["a_scale"]) @ scaled_blocks(s["b"], s["b_scale"]).T).to(torch.bfloat16)}
    if op == "grouped":
        a, group, at = padded_groups(s, scaled_rows(s["a"], s["a_scale"]))
        out = torch.bmm(a, scaled_blocks(s["b"], s["b_scale"]).transpose(1, 2))
        return {"out": out[group, at].to(torch.bfloat16)}
    dy, x = s["dy"].float(), s["x"].float()
    dq = scaled_rows(*quantised_rows(dy))
    w = scaled_blocks(s["b"], s["b_scale"])
    if op == "gemm_back":
        return {"dx": (dq @ w.T).to(torch.bfloat16), "dw": plain_weight_gradient(dy, x)}
    a, group, at = padded_groups(s, dq)
    dx = torch.bmm(a, w.transpose(1, 2))[group, at]
    return {"dx": dx.to(torch.bfloat16), "dw": plain_weight_gradient(padded_groups(s, dy)[0], padded_groups(s, x)[0])}


# ------------------------------------------------------- the library's calls --

def library(s):
    from dense_int8_matrix_gb300 import binding as B
    op = s["op"]
    if op == "norm_f8":
        B.gemm_norm_f8(s["x"], s["r"], s["w"], EPS, s["h"], s["rstd"], s["q"], s["scale"])
        return {"h": s["h"], "rstd": s["rstd"], "q": s["q"], "scale": s["scale"]}
    if op == "norm_i8":
        B.gemm_norm_i8(s["x"], s["r"], s["w"], EPS, s["h"], s["rstd"], s["q"], s["scale"])
        B.gemm_i8_run_requant(s["plan"], s["q"], s["wt"], s["scale"], s["col_scale"], s["out"])
        return {"h": s["h"], "rstd": s["rstd"], "scale": s["scale"], "out": s["out"]}
    if op == "norm_back":
        B.gemm_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], s["dr"], s["dx"], s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "gemm":
        B.gemm_f8_run(s["plan"], s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"])
        return {"out": s["out"]}
    if op == "grouped":
        B.gemm_f8_grouped_run(s["plan"], s["a"], s["a_scale"], s["b"], s["b_scale"], s["offsets"], s["out"])
        return {"out": s["out"]}
    off = s.get("offsets")
    B.gemm_f8_quantize(s["dy"], s["dy_q"], s["dy_s"])
    B.gemm_f8_quantize_cols(s["dy"], s["dy_qc"], s["dy_sc"], off)
    B.gemm_f8_quantize_cols(s["x"], s["x_qc"], s["x_sc"], off)
    if op == "gemm_back":
        B.gemm_f8_run(s["plan"], s["dy_q"], s["dy_s"], s["b"], s["b_scale"], s["dx"])
        B.gemm_f8_run(s["plan_w"], s["dy_qc"], s["dy_sc"], s["x_qc"], s["x_sc"], s["dw"])
    else:
        B.gemm_f8_grouped_run(s["plan"], s["dy_q"], s["dy_s"], s["b"], s["b_scale"], off, s["dx"])
        B.gemm_f8_grouped_run(s["plan_w"], s["dy_qc"], s["dy_sc"], s["x_qc"], s["x_sc"], off, s["dw"])
    return {"dx": s["dx"], "dw": s["dw"]}


def run(state):
    return library(state) if own else plain(state)


# ---------------------------------------------------------- work, and truth --

def work(case):
    op = case["op"]
    if op in ("norm_f8", "norm_i8", "norm_back"):
        rows, d = case["rows"], case["d"]
        if op == "norm_f8":     # x, r, h at 2 bytes, q at 1, scales, rstd, w
            return {"bytes": 7 * rows * d + 4 * rows * (blocks_of(d) + 1) + 4 * d, "flops": 10 * rows * d}
        if op == "norm_i8":     # x, r, h, the int8 weights, the product
            n = case["n"]
            return {"bytes": 6 * rows * d + n * d + 2 * rows * n + 4 * (2 * rows + d + n), "flops": 2 * rows * d * n + 10 * rows * d}
        return {"bytes": 8 * rows * d + 4 * rows + 8 * d, "flops": 12 * rows * d}   # dy, h, dr, dx; w, dw
    m, k, n, groups = case["m"], case["k"], case["n"], case.get("groups", 1)
    mn, mk, nk = m * n, m * k, n * k * (min(groups, m) if op == "grouped" else groups)
    if op in ("gemm", "grouped"):
        return {"bytes": mk + nk + 2 * mn + 4 * (m * blocks_of(k) + nk // BLOCK ** 2 + groups), "flops": 2 * mn * k}
    # dY and X at 2 bytes, the weights at 1, dX at 2, dW at 4
    return {"bytes": 2 * mn + 2 * mk + nk + 2 * mk + 4 * nk, "flops": 4 * mn * k}


def truth_quantised(x):
    """The e4m3 blocks of 128 columns in 64 bits: the values before rounding, the scales, the values after."""
    rows, k = x.shape
    kb = -(-k // 128)
    full = torch.zeros(rows, kb * 128, dtype=torch.float64, device=x.device)
    full[:, :k] = x
    full = full.view(rows, kb, 128)
    scale = torch.clamp(full.abs().max(dim=2).values / 448.0, min=2.0 ** -126)
    codes = full / scale.float().double()[:, :, None]
    near = codes.float().to(torch.float8_e4m3fn).double() * scale[:, :, None]
    return codes.reshape(rows, -1)[:, :k], scale, near.reshape(rows, -1)[:, :k]


def truth_values(q, scale, rows_per_scale):
    out = q.double()
    for b in range(0, q.shape[1], 128):
        sc = scale[:, b // 128].double()
        if rows_per_scale > 1:
            sc = sc.repeat_interleave(rows_per_scale)[: q.shape[0]]
        out[:, b : b + 128] *= sc[:, None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm_f8", "norm_i8"):
        h = (s["x"].double() + s["r"].double()).to(torch.bfloat16)
        hd = h.double()
        rstd = 1.0 / torch.sqrt(torch.einsum("ij,ij->i", hd, hd) / case["d"] + EPS)
        y = hd * s["w"].double() * rstd[:, None]
        if op == "norm_f8":
            codes, scale, _ = truth_quantised(y)
            return {"h": hd, "rstd": rstd, "q": codes, "scale": scale.T.contiguous()}
        scale = y.abs().max(dim=1).values / 127.0
        q = torch.round(y / scale[:, None])
        return {"h": hd, "rstd": rstd, "scale": scale,
                "out": torch.einsum("ij,kj->ik", q, s["wt"].double()) * scale[:, None] * s["col_scale"].double()[None, :]}
    if op == "norm_back":
        h, dy, w, r = s["h"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()
        dot = torch.einsum("ij,ij,j->i", dy, h, w) / case["d"]
        dx = s["dr"].double() + dy * w * r[:, None] - h * (r ** 3 * dot)[:, None]
        return {"dx": dx, "dw": torch.einsum("ij,ij,i->j", dy, h, r)}
    ends = s["offsets"].tolist() if "offsets" in s else [0, case["m"]]
    b = s["b"] if "offsets" in s else s["b"][None]
    bs = s["b_scale"] if "offsets" in s else s["b_scale"][None]
    if op in ("gemm", "grouped"):
        a = truth_values(s["a"], s["a_scale"].T, 1)
    else:
        a = truth_quantised(s["dy"].double())[2]
    out = torch.cat([a[lo:hi] @ truth_values(b[i], bs[i], 128).T for i, (lo, hi) in enumerate(zip(ends, ends[1:]))])
    if op in ("gemm", "grouped"):
        return {"out": out}
    dw = [truth_quantised(s["dy"][lo:hi].double().T)[2] @ truth_quantised(s["x"][lo:hi].double().T)[2].T if hi > lo
          else torch.zeros(case["n"], case["k"], dtype=torch.float64, device="cuda") for lo, hi in zip(ends, ends[1:])]
    return {"dx": out, "dw": torch.stack(dw) if "offsets" in s else dw[0]}
