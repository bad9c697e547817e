"""A norm's gradients against differences of its outputs, with tolerances that are derived and small.

The weighted sum of a row, S(x) = sum over c of dy_c y_c, is w . u r + a constant, with w = dy gamma,
u = x (rms) or x less its mean (layer), q = |u|^2 / n + eps and r = q^(-1/2).  Along directions d and e
|q_d| <= 2 |d| (q/n)^(1/2), |q_de| <= 2 |d||e| / n and |u| <= (n q)^(1/2), so that
  |r_d|  <= |d| n^(-1/2) / q,   |r_de| <= 4 |d||e| q^(-3/2) / n,   |r_ddd| <= 24 |d|^3 q^(-2) n^(-3/2),
  |S_de|  <= |w||u||r_de| + |w||d||r_e| + |w||e||r_d|  <= 6 |w||d||e| n^(-1/2) / q,
  |S_ddd| <= |w||u||r_ddd| + 3 |w||d||r_dd|            <= 36 |w||d|^3 q^(-3/2) / n.
The quotient (S(x + d) - S(x - d)) / 2 is off from S_d by at most a sixth of the largest |S_ddd| between
the two points, where q^(1/2) is at least its value in the middle less |d| n^(-1/2).

The gradients start from the forward pass's mean and r in fp32: off by m and, relative to r, by p at most,
they move h by a vector g of at most p |h| + n^(1/2) m r.  That moves c2 by at most |a||g| / n, dx along d
by at most p |dx . d| + r |d| (|g||c2| + |h||a||g| / n), and dgamma along e by the rows' |dy e||g|."""

import torch

import layer_ref as ref


def inputs(rows, cols, seed):
    """x, dy, gamma, beta in fp32; dy has a mean and a part along x, so that c1 and c2 are of its size."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = n(rows, cols) + 0.3
    return x, n(rows, cols) + 0.5 + 0.5 * x, 1.0 + 0.2 * n(cols), 0.2 * n(cols)


def mid(up, down):
    """Both points' middle and half their difference, in 64 bits."""
    return (up.double() + down.double()) / 2, (up.double() - down.double()) / 2


def check(forward, x, dy, gamma, beta, kind, eps, dx, dgamma, dbeta):
    """forward(x, gamma, beta) -> y in fp32, on the CPU; dx, dgamma and dbeta in fp32, from the forward
    pass's statistics: what is checked, each row of dx for itself.  Raises AssertionError."""
    rows, n = x.shape
    wide = [t.double() for t in (dy, x, gamma, beta)]
    mean = wide[1].mean(1) if kind == "layer" else None
    u = wide[1] - (mean[:, None] if kind == "layer" else 0.0)
    q = (u * u).sum(1) / n + eps
    none = torch.zeros(rows, n, dtype=torch.float64)
    own = ref.norm_grad(wide[0], wide[1], mean, q.rsqrt(), wide[2], none, kind, torch.float32, torch.float32,
                        none[0], none[0])
    stats = ref.norm(wide[1], wide[2], wide[3], kind, eps, torch.float32)
    p = stats["rstd"][1] / stats["rstd"][0]
    h, a = u * q.rsqrt()[:, None], wide[0] * wide[2]
    g = p * h.norm(dim=1)
    if kind == "layer":
        g = g + n ** 0.5 * stats["mean"][1] * q.rsqrt()
    g = ref.SLACK * g

    def sums(x, gamma, beta):
        """The weighted sums of y, and how far rounding may put them off."""
        bound = ref.norm(x.double(), gamma.double(), beta.double(), kind, eps, torch.float32)["y"][1]
        return wide[0] * forward(x, gamma, beta).double(), wide[0].abs() * bound

    # dx: a direction with parts along the gradient, the ones and the row, each of which c1 or c2 takes off
    unit = lambda t: t / t.norm(dim=1, keepdim=True)  # noqa: E731
    d = (0.25 * unit(unit(own["dx"][0]) + unit(torch.ones_like(u)) + unit(u))).float()
    up, down = x + d, x - d
    (s1, b1), (s0, b0) = sums(up, gamma, beta), sums(down, gamma, beta)
    middle, d = mid(up, down)
    size, w = d.norm(dim=1), a.norm(dim=1)
    root = q.sqrt() - (size + (middle - wide[1]).norm(dim=1)) / n ** 0.5
    off = (b1 + b0).sum(1) / 2 + 36 / 6 * w * size ** 3 / root ** 3 / n \
        + 6 * w * size * (middle - wide[1]).norm(dim=1) / n ** 0.5 / root ** 2 \
        + (own["dx"][1] * d.abs()).sum(1) + p * (own["dx"][0] * d).sum(1).abs() \
        + q.rsqrt() * size * g * ((a * h).mean(1).abs() + h.norm(dim=1) * w / n)
    got, want = (dx.double() * d).sum(1), ((s1 - s0) / 2).sum(1)
    assert float((off / want.abs()).max()) < 0.02, "the tolerance is no small part of the derivative"
    assert float(((got - want).abs() / off).max()) <= 1.0, "dx"

    # the weights': y is linear in them, so the quotient is exact but for rounding, and the direction may be long
    for name, i, value in (("dgamma", 0, dgamma), ("dbeta", 1, dbeta)):
        both = []
        of_stats = lambda d: float(((wide[0] * d).norm(dim=1) * g).sum()) if i == 0 else 0.0  # noqa: E731
        e = own[name][0].float() / float(own[name][0].norm())
        for sign in (1.0, -1.0):
            args = [gamma, beta]
            args[i] = args[i] + sign * e
            both.append((args[i], *sums(x, *args)))
        (up, s1, b1), (down, s0, b0) = both
        d = mid(up, down)[1]
        off = float((b1 + b0).sum() / 2 + (own[name][1] * d.abs()).sum()) + of_stats(d)
        got, want = float((value.double() * d).sum()), float(((s1 - s0) / 2).sum())
        assert off < 0.02 * abs(want), "the tolerance is no small part of the derivative"
        assert abs(got - want) <= off, name
