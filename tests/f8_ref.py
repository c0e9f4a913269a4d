"""64-bit references of the 8-bit operators and seeded inputs for their tests
(numpy and torch on the CPU; none of the library's code)."""

from __future__ import annotations

import torch

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
MAXIMUM = {E4M3: 448.0, E5M2: 57344.0}
SCALE_MIN = 2.0 ** -126


def gen(seed: int) -> torch.Generator:
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


def pad16(k: int) -> int:
    return (k + 15) // 16 * 16


def padded_k(rows: int, groups: int) -> int:
    return (rows + 127 * groups) // 128 * 128


def whole_f8(shape, seed, dtype=E4M3, most=8):
    """Whole numbers in [-most, most] as FP8 (exact in both types for most <= 8)."""
    return torch.randint(-most, most + 1, shape, generator=gen(seed)).float().to(dtype)


def normal_f8(shape, seed, dtype=E4M3):
    """N(0, 1) scaled so that the largest values reach well into the type's range."""
    return (torch.randn(shape, generator=gen(seed)) * 60.0).to(dtype)


def power_scales(shape, seed):
    return torch.exp2(torch.randint(-2, 3, shape, generator=gen(seed)).float())


def any_scales(shape, seed):
    return torch.rand(shape, generator=gen(seed)) * 0.02 + 1e-4


def expand_rows(scale, k):
    """(kb, rows) -> (rows, k)."""
    return scale.double().T.repeat_interleave(128, 1)[:, :k]


def expand_blocks(scale, n, k):
    """(nb, kb) -> (n, k)."""
    return scale.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def product(A, a_full, Bt, b_full):
    """(D, S) in 64 bits: the product of the scaled values, and the sum of the terms' magnitudes."""
    a, b = A.float().double() * a_full, Bt.float().double() * b_full
    return a @ b.T, a.abs() @ b.abs().T


def padded_starts(sizes):
    """First padded column of each group, and the end."""
    at = [0]
    for s in sizes:
        at.append(at[-1] + (s + 127) // 128 * 128)
    return at


def scale_of(amax, dtype):
    """fp32 scale of a block (fp32 arithmetic, as the operator is defined)."""
    step = torch.tensor(1.0) / torch.tensor(MAXIMUM[dtype])   # the reciprocal, rounded to fp32
    return torch.clamp_min(amax.float() * step, SCALE_MIN)


def quantised(x, scale_full, dtype):
    """x * (1 / scale) in fp32 steps, rounded to the FP8 type."""
    m = MAXIMUM[dtype]
    return (x.float() * (1.0 / scale_full.float())).clamp(-m, m).to(dtype)


def quantise_rows(x, dtype):
    """(q, scale (kb, rows)) of 1 x 128 blocks."""
    rows, k = x.shape
    kb = (k + 127) // 128
    xp = torch.zeros(rows, kb * 128)
    xp[:, :k] = x.float()
    s = scale_of(xp.view(rows, kb, 128).abs().amax(2), dtype)
    return quantised(x, s.repeat_interleave(128, 1)[:, :k], dtype), s.T.contiguous()


def quantise_blocks(x, dtype):
    rows, k = x.shape
    rb, kb = (rows + 127) // 128, (k + 127) // 128
    xp = torch.zeros(rb * 128, kb * 128)
    xp[:rows, :k] = x.float()
    s = scale_of(xp.view(rb, 128, kb, 128).abs().amax((1, 3)), dtype)
    full = s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :k]
    return quantised(x, full, dtype), s


def norm(x, r, w, eps, dtype):
    """(h, rstd, y): h rounded to dtype, the others in 64 bits."""
    h = (x.double() + (r.double() if r is not None else 0.0)).to(dtype)
    hd = h.double()
    rstd = 1.0 / torch.sqrt(hd.square().mean(1) + eps)
    return h, rstd, hd * rstd[:, None] * w.double()


def norm_backward(dy, h, w, rstd, dr):
    dy, h, w, rstd = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    xhat, g = h * rstd, dy * w
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    return dx + (dr.double() if dr is not None else 0.0), (dy * xhat).sum(0)
