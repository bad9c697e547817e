"""Plain numpy references of the AdamW operators, for the GPU tests.

Two of each: the stated fp32 sequence, one rounded operation at a time (the
library is bit-identical to it), and the definition in 64 bits, with bounds on
how far the fp32 sequence may be from it.  Both share no code with the library.
"""

from __future__ import annotations

import numpy as np

F = np.float32
U = 2.0 ** -24  # half a step of fp32, relative
BLOCK = 256
TOP = {"m": 448.0, "v": 57344.0}
LEAST = {"m": -6, "v": -14}  # exponent of the smallest normal value
BITS = {"m": 3, "v": 2}      # fraction bits


def scale_of(grad_scale, sumsq=None, max_norm=0.0):
    """(gs as a double, norm finite)."""
    if sumsq is None:
        return grad_scale, True
    with np.errstate(all="ignore"):
        norm = float(np.sqrt(np.float64(sumsq)) * abs(grad_scale))
        coef = 1.0
        if max_norm > 0:
            coef = float(np.float64(max_norm) / (np.float64(norm) + 1e-6))
            coef = 1.0 if coef > 1.0 else coef
    return grad_scale * coef, bool(np.isfinite(norm))


def mean32(grads):
    """Left fold over the ranks in fp32, over their number."""
    s = grads[0].astype(F)
    for g in grads[1:]:
        s = s + g.astype(F)
    return s if len(grads) == 1 else s / F(len(grads))


def step32(g, w, m, v, h, bits=32):
    """One step of the fp32 sequence from the mean gradient; h: dict of lr (the
    tensor's), decay, beta1, beta2, eps, step, gs.  Returns (w, m, v) and, for
    8 bits, how far the hardware's root and reciprocal may take w from here:
    relative to u, root 2 U (1 ulp) + U here, its constant, product and sum 3 U
    on each side, reciprocal 2 U, product U and the folded constant U against
    the constant, product and quotient 3 U here: under 18 U; then a product and
    two sums on each side, U of each one's result."""
    b1, b2, t = h["beta1"], h["beta2"], h["step"]
    bc1, bc2 = 1.0 - b1 ** t, 1.0 - b2 ** t
    with np.errstate(all="ignore"):
        g = g * F(h["gs"])
        m = F(b1) * m + F(1.0 - b1) * g
        v = F(b2) * v + F(1.0 - b2) * (g * g)
        if bits == 32:
            u = (m / F(bc1)) / (np.sqrt(v / F(bc2)) + F(h["eps"]))
        else:
            u = (m * F(1.0 / bc1)) / (np.sqrt(v) * F(1.0 / np.sqrt(bc2)) + F(h["eps"]))
        lu, lw = F(h["lr"]) * u, F(h["lr"] * h["decay"]) * w
        w = w - (lu + lw)
        if bits == 32:
            return w, m, v
        off = U * (22.0 * np.abs(lu).astype(np.float64) + 4.0 * np.abs(lw) + 2.1 * np.abs(w))
    return w, m, v, off


def step64(grads, w, m, v, h, bits=32):
    """The definition in 64 bits and bounds on the fp32 sequence's distance:
    (w, m, v, bw, bm, bv).  Each operation, constant and sum in fp32 is off by
    at most U relative (no product here underflows: the tests' values do not)."""
    b1, b2, t, p = h["beta1"], h["beta2"], h["step"], len(grads)
    g = sum(x.astype(np.float64) for x in grads) / p
    size = sum(np.abs(x.astype(np.float64)) for x in grads) / p
    g, size = g * h["gs"], size * abs(h["gs"])
    # p-1 additions, a division, the factor's rounding and its product
    bg = (p + 2) * U * size
    w, m, v = (x.astype(np.float64) for x in (w, m, v))
    m2 = b1 * m + (1 - b1) * g
    # each product: the constant's rounding and its own; then the sum's
    bm = (1 - b1) * bg + 3.1 * U * (np.abs(b1 * m) + (1 - b1) * (np.abs(g) + bg))
    v2 = b2 * v + (1 - b2) * g * g
    bv = (1 - b2) * (2 * np.abs(g) + bg) * bg + 4.1 * U * (b2 * v + (1 - b2) * (np.abs(g) + bg) ** 2)
    mh, vh = m2 / (1 - b1 ** t), v2 / (1 - b2 ** t)
    d = np.sqrt(vh) + h["eps"]
    u = mh / d
    # m_hat: the constant and a division; the root: half of v's relative error, the constant, two roundings,
    # the sum with eps (eps rounded too); then the quotient
    rel_d = np.divide(bv, 2 * v2, out=np.zeros_like(v2), where=v2 > 0) * (1 + 1e-3) + 5.1 * U
    if bits == 8:  # a root of 1 ulp (2 U), and a reciprocal of 1 ulp and a product for the quotient
        rel_d += 1.1 * U
    bu = bm / (1 - b1 ** t) / d + np.abs(u) * (rel_d + (3.1 if bits == 32 else 5.1) * U)
    lr, ld = h["lr"], h["lr"] * h["decay"]
    w2 = w - (lr * u + ld * w)
    bw = abs(lr) * bu + 3.2 * U * (np.abs(lr * u) + np.abs(ld * w)) + 1.1 * U * np.abs(w2)
    return w2, m2, v2, bw, bm, bv


def philox(index, step, seed):
    """Philox4x32-7 of (index, step) under seed: four uint32 words per index."""
    word = np.uint64(0xFFFFFFFF)
    c = [np.asarray(index, np.uint64) & word, np.asarray(index, np.uint64) >> np.uint64(32)]
    c += [np.full_like(c[0], step & 0xFFFFFFFF), np.full_like(c[0], step >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(7):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & word,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & word]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack([x.astype(np.uint32) for x in c], -1)


def grid_values(kind):
    """What the 256 codes stand for (OCP e4m3 without infinities, e5m2 with)."""
    c = np.arange(256)
    e, f = (c & 127) >> BITS[kind], c & ((1 << BITS[kind]) - 1)
    n = 1 << BITS[kind]
    x = np.where(e == 0, f / n * 2.0 ** LEAST[kind], (1 + f / n) * 2.0 ** (e - 1.0 + LEAST[kind]))
    if kind == "m":
        x[(c & 127) == 127] = np.nan
    else:
        x[(c & 127) == 124] = np.inf
        x[(c & 127) > 124] = np.nan
    return np.where(c & 128, -x, x)


def code_of(values, kind):
    """Codes of values that lie on the grid."""
    grid = grid_values(kind)[:128]
    grid = grid[np.isfinite(grid)]
    a = np.abs(values).astype(np.float64)
    c = np.searchsorted(grid, a)
    assert np.array_equal(grid[c], a)
    return (c | np.where(np.signbit(values), 128, 0)).astype(np.uint8)


def encode(x, kind, halves=None):
    """(codes, scales) of fp32 values, in the stated fp32 sequence; halves: 16
    random bits per value, or None for rounding to nearest even."""
    n = x.size
    nb = -(-n // BLOCK)
    y = np.zeros(nb * BLOCK, F)
    y[:n] = x
    y = y.reshape(nb, BLOCK)
    live_at = F(2.0 ** -110)
    scales = np.zeros(nb, F)
    codes = np.zeros((nb, BLOCK), np.uint8)
    top = F(TOP[kind])
    if halves is not None:
        h = np.zeros(nb * BLOCK, np.uint32)
        h[:n] = halves
        h = h.reshape(nb, BLOCK)
    for b in range(nb):
        row = y[b]
        if not np.all(np.isfinite(row)):
            scales[b] = np.nan
            continue
        most = np.abs(row).max()
        if most < live_at:
            continue
        scales[b] = most * F(1.0 / TOP[kind])
        z = np.clip(row * (top / most), -top, top)
        if halves is None:
            a = np.abs(z).astype(np.float64)
            e = np.maximum(np.frexp(a)[1] - 1, LEAST[kind])
            q = np.ldexp(1.0, e - BITS[kind])
            z = np.copysign(np.round(a / q) * q, z)
        else:
            cut = 23 - BITS[kind]
            least = F(2.0 ** LEAST[kind])
            a = np.abs(z)
            low = a < least
            a = np.where(low, a + least, a)
            r = (h[b].astype(np.uint32) << np.uint32(cut - 16)) + np.uint32(1 << (cut - 17))
            a = ((a.view(np.uint32) + r) & np.uint32(0xFFFFFFFF ^ ((1 << cut) - 1))).view(F)
            z = np.copysign(np.where(low, a - least, a), z)
        c = code_of(z, kind)
        if kind == "v":
            c = np.where((row > 0) & ((c & 127) == 0), 1, c).astype(np.uint8)
        codes[b] = c
    return codes.reshape(-1)[:n], scales


def decode(codes, scales, kind):
    n = codes.size
    with np.errstate(all="ignore"):
        return grid_values(kind).astype(F)[codes] * np.repeat(scales, BLOCK)[:n]


def halves_for(n, index, step, seed):
    """(low, high) 16 random bits of each of a tensor's n values."""
    nq = -(-n // 4)
    w = philox(np.uint64(index) + 4 * np.arange(nq, dtype=np.uint64), step, seed).reshape(-1)[:n]
    return w & np.uint32(0xFFFF), w >> np.uint32(16)
