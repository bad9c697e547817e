"""The layer operators in 64 bits, written from their formulas, with bounds on how
far fp32 arithmetic in the stated operations may be off, for any order of the
sums.

U is the most that one fp32 operation is off, relative to its result.  A sum of
terms x that any of which passes through k additions is off by at most about
k * U * sum |x|.  Products of small errors are covered by the factor SLACK.
"""

import torch

U = 2.0 ** -24
SLACK = 1.02
# Additions that an element of a row passes through: 16 in its lane, 6 steps over
# the wave, 16 waves, and the division.
ROW_ADDS = 40
TD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def column_adds(rows):
    """The same for a sum over rows.  A lane adds those of its own turns: a 128th of
    the rows at most where a launch has all 256 CUs' workgroups, and of 1024 rows at
    most where few are read by columns, a 64th, 16.  Then come at most 16 waves, or
    32 teams (of 16 lanes), and 512 parts by 64 in 8 turns and in 6 steps: 46 of the
    64 here."""
    return min(rows, rows // 128 + 1) + 16 + 16 + 32


def rounding(y, dtype):
    """Half a step of the type at y (half the smallest subnormal near 0)."""
    f = torch.finfo(dtype)
    return (y.abs() * (f.eps / 2)).clamp(min=f.smallest_normal * f.eps / 2)


def norm(t, gamma, beta, kind, eps, dtype):
    """t, gamma, beta in 64 bits -> {name: (value, bound)}."""
    n = t.shape[1]
    mean, e_mean = torch.zeros(t.shape[0], dtype=torch.float64), 0.0
    if kind == "layer":
        mean = t.sum(1) / n
        e_mean = (ROW_ADDS + 1) * U * t.abs().sum(1) / n
    d = t - mean[:, None]
    e_d = (e_mean[:, None] + U * d.abs()) if kind == "layer" else torch.zeros_like(d)
    var = (d * d).sum(1) / n
    e_var = (2 * d.abs() * e_d + e_d * e_d).sum(1) / n + (ROW_ADDS + 2) * U * var
    # of the sum with eps, the root and the division
    rel = e_var / (2 * (var + eps)) * SLACK + 3 * U
    rstd = 1 / torch.sqrt(var + eps)
    h = d * rstd[:, None]
    e_h = e_d * rstd[:, None] + h.abs() * (rel + U)[:, None]
    y = h * gamma + beta
    e_y = e_h * gamma.abs() + 2 * U * (h * gamma).abs() + U * y.abs()
    out = {"y": (y, SLACK * e_y + rounding(y, dtype)), "rstd": (rstd, SLACK * rel * rstd)}
    if kind == "layer":
        out["mean"] = (mean, SLACK * e_mean + U * mean.abs())
    return out


def norm_grad(dy, x, mean, rstd, gamma, dres, kind, dtype, gdtype, old_gamma, old_beta):
    """All in 64 bits; dres and the old gradients may be zeros."""
    rows, n = x.shape
    layer = kind == "layer"
    h = (x - mean[:, None] if layer else x) * rstd[:, None]
    e_h = (2 if layer else 1) * U * h.abs()
    a = dy * gamma
    c1 = a.sum(1, keepdim=True) / n if layer else torch.zeros(rows, 1, dtype=torch.float64)
    c2 = (a * h).sum(1, keepdim=True) / n
    e1 = (ROW_ADDS + 2) * U * a.abs().sum(1, keepdim=True) / n if layer else 0.0
    e2 = (ROW_ADDS + 5) * U * (a * h).abs().sum(1, keepdim=True) / n
    inner = a - c1 - h * c2
    e = U * a.abs() + e1 + U * (a - c1).abs() + e2 * h.abs() + c2.abs() * e_h + U * (h * c2).abs() \
        + 2 * U * inner.abs()
    dx = inner * rstd[:, None] + dres
    e_dx = e * rstd[:, None] + U * dx.abs()
    k = column_adds(rows)
    out = {"dx": (dx, SLACK * e_dx + rounding(dx, dtype))}
    terms = dy * h
    for name, x64, old, own in (("dgamma", terms, old_gamma, 3), ("dbeta", dy, old_beta, 0)):
        s = x64.sum(0) + old
        e_s = (k + own) * U * x64.abs().sum(0) + U * s.abs()
        out[name] = (s, SLACK * e_s + rounding(s, gdtype))
    return out


def embed_grad(dy, row, rows, scale, old, gdtype):
    """dy in 64 bits, row: each token's row or -1; old: what is added to, or zeros."""
    cols = dy.shape[1]
    inside = row >= 0
    at, x = row[inside], dy[inside]
    sums = torch.zeros(rows, cols, dtype=torch.float64).index_add_(0, at, x)
    sizes = torch.zeros(rows, cols, dtype=torch.float64).index_add_(0, at, x.abs())
    count = torch.zeros(rows, dtype=torch.float64).index_add_(
        0, at, torch.ones(len(at), dtype=torch.float64))
    y = sums * scale + old
    e = (count + 1)[:, None] * U * sizes * abs(scale) + U * (sums * scale).abs() + U * y.abs()
    return y, SLACK * e + rounding(y, gdtype), count
