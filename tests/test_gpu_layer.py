"""The layer operators on the GPU against the 64-bit references of layer_ref, within
the bounds that it derives; exactly where a result has one value only."""

import numpy as np
import pytest
import torch

import layer_diff
import layer_ref as ref
from adam_zs_shard_amd import zsadamw as aw
from adam_zs_shard_amd import zslayer as a
from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
TD = ref.TD
EPS = 1e-5


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Buf:
    """rows x cols elements in a flat buffer of canaries: `shift` elements in, `gap` between two rows."""

    CANARY = {4: 0x5A5A5A5A, 2: 0x5A5A}

    def __init__(self, rows, cols, dtype, shift=0, gap=0, values=None):
        self.dtype, size = dtype, torch.empty(0, dtype=dtype).element_size()
        raw = {4: torch.int32, 2: torch.int16}[size]
        n = shift + rows * (cols + gap) + 64
        self.flat = torch.full((n,), self.CANARY[size], dtype=raw, device=DEV)
        self.own = torch.zeros(n, dtype=torch.bool, device=DEV)
        self.t = self._cut(self.flat.view(dtype), rows, cols, shift, gap)
        self._cut(self.own, rows, cols, shift, gap)[:] = True
        self.raw, self.size = raw, size
        if values is not None:
            self.t.copy_(values)

    @staticmethod
    def _cut(x, rows, cols, shift, gap):
        return x.as_strided((rows, cols), (cols + gap, 1), shift)

    def check(self, what):
        assert bool((self.flat[~self.own] == self.CANARY[self.size]).all()), f"{what}: written outside"

    def cpu64(self):
        return self.t.detach().cpu().double()


def within(got, value_bound, what):
    value, bound = value_bound
    got = got.detach().cpu().double().reshape(value.shape)
    far = (got - value).abs() / bound
    assert torch.isfinite(got).all(), what
    worst = float(far.max()) if far.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def garbage(nbytes):
    """A workspace of NaN, whatever it is read as."""
    return torch.full((max(nbytes, 1),), 0xFF, dtype=torch.uint8, device=DEV)


def activations(rows, cols, seed):
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g) * (0.2 + 2 * torch.rand(rows, 1, generator=g))
    x += 0.5 * torch.randn(rows, 1, generator=g)
    x[:, :: 97] *= 15
    return x


def weights(cols, wdt, seed, present):
    g = gen(seed)
    return [(m + 0.2 * torch.randn(cols, generator=g)).to(TD[wdt]).to(DEV) if p else None
            for m, p in zip((1.0, 0.0), present)]


def wide(w, cols, none):
    return torch.full((cols,), none, dtype=torch.float64) if w is None else w.cpu().double()


# ----------------------------------------------------------------- the norm

COLS = [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 768, 1000, 1023, 1024, 1025, 2047, 2048, 2050, 4095, 4096,
        4097, 5120, 8191, 8192, 8193, 12289, 16383, 16384]


def run_norm(rows, cols, kind, dt, wdt="bf16", residual=False, shift=0, gap=0, present=(True, True), eps=EPS,
             seed=0, x=None, place=None):
    dtype = TD[dt]
    x = activations(rows, cols, seed) if x is None else x
    X = Buf(rows, cols, dtype, shift, gap, x)
    R = Buf(rows, cols, dtype, shift + 1, 2 * gap, torch.randn(rows, cols, generator=gen(seed + 1))) \
        if residual else None
    x64 = X.cpu64()
    T = {None: Buf(rows, cols, dtype, shift, gap) if residual else None, "total=x": X, "total=residual": R,
         "y=x": Buf(rows, cols, dtype, shift, gap) if residual else None}[place]
    Y = X if place == "y=x" else Buf(rows, cols, dtype, 2 * shift, gap)
    gamma, beta = weights(cols, wdt, seed + 2, present)
    mean = Buf(1, rows, torch.float32) if kind == "layer" else None
    rstd = Buf(1, rows, torch.float32)
    if residual:
        t = (X.t.float() + R.t.float()).to(dtype).cpu()      # one rounding each way
    a.zs_norm_forward(rows, cols, X.t, Y.t, gamma, beta, kind=kind, eps=eps, residual=R.t if R else None,
                      total=T.t if T else None, mean=mean.t if mean else None, rstd=rstd.t,
                      w_dtype=wdt if any(present) else None)
    t64 = x64
    if residual:
        assert torch.equal(T.t.cpu(), t)
        t64 = t.double()
    want = ref.norm(t64, wide(gamma, cols, 1.0), wide(beta, cols, 0.0), kind, float(np.float32(eps)), dtype)
    within(Y.t, want["y"], "y")
    within(rstd.t, want["rstd"], "rstd")
    if mean:
        within(mean.t, want["mean"], "mean")
    for b in (X, R, T, Y, mean, rstd):
        if b:
            b.check("buffer")


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_norm_of_every_width(kind, dt):
    for i, cols in enumerate(COLS):
        run_norm(5, cols, kind, dt, seed=i)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 4096), (2, 768), (3, 100), (4, 64), (5, 2048), (1000, 33), (777, 768),
                                       (9001, 40), (4100, 600), (1037, 5000), (600, 16384)])
def test_norm_of_many_rows(rows, cols, dt):
    run_norm(rows, cols, "layer", dt, residual=True, seed=rows)
    run_norm(rows, cols, "rms", dt, seed=rows)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt,wdt", [("bf16", "f32"), ("f16", "bf16"), ("f32", "f16"), ("f32", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("shift,gap", [(1, 0), (3, 5), (8, 8), (2, 1)])
def test_norm_at_odd_places(kind, dt, wdt, shift, gap):
    for cols in (31, 768, 1001, 4100):
        run_norm(6, cols, kind, dt, wdt, residual=True, shift=shift, gap=gap, seed=cols)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("present", [(False, False), (True, False), (False, True)])
def test_norm_without_weights(kind, present):
    run_norm(7, 500, kind, "bf16", present=present)
    run_norm(7, 3000, kind, "f32", present=present, residual=True)


@pytest.mark.parametrize("place", ["total=x", "total=residual", "y=x"])
@pytest.mark.parametrize("cols", [100, 768, 6000])
def test_norm_in_place(place, cols):
    run_norm(50, cols, "layer", "bf16", residual=True, gap=4 * (place != "total=residual"), place=place)
    if place == "y=x":
        run_norm(50, cols, "rms", "f16", place=place)


# teams of 16, 32 and 64 lanes, whole and broken waves and workgroups of them
NARROW = [(1, 128), (3, 64), (5, 129), (17, 127), (31, 256), (33, 255), (63, 128), (1025, 192), (4097, 257),
          (20_000, 128), (33_000, 65), (9000, 512)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", NARROW)
def test_norm_of_narrow_rows(rows, cols, dt):
    run_norm(rows, cols, "layer", dt, "f32", residual=True, gap=cols, seed=rows)
    run_norm(rows, cols, "rms", dt, seed=rows, place="y=x")


REMAINDERS = [*range(1, 25), *range(1040, 1048)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", REMAINDERS)
def test_norm_of_every_remainder(cols, dt):
    run_norm(9, cols, "layer", dt, "f16", residual=True, shift=1, gap=1, seed=cols)
    run_norm(9, cols, "rms", dt, "f32", residual=True, gap=2, place="total=x", seed=cols)


def test_norm_of_columns_of_one_buffer():
    """Input and output side by side in the same rows."""
    b = torch.randn(9, 3 * 700, generator=gen(3)).bfloat16().to(DEV)
    x, keep, y = b[:, :700], b[:, 700:1400].clone(), b[:, 1400:]
    before = x.clone()
    a.zs_norm_forward(9, 700, x, y, kind="rms", eps=EPS)
    want = ref.norm(before.cpu().double(), torch.ones(700).double(), torch.zeros(700).double(), "rms",
                    float(np.float32(EPS)), torch.bfloat16)
    within(y, want["y"], "y")
    assert torch.equal(x, before) and torch.equal(b[:, 700:1400], keep)


def test_norm_of_a_large_mean():
    """A mean 1000 times the spread: the difference of two sums would have no digit left."""
    x = 4096.0 + torch.randn(20, 2000, generator=gen(5))
    run_norm(20, 2000, "layer", "f32", x=x, present=(True, True))


def test_norm_of_equal_values_and_of_zeros():
    x = torch.cat([torch.full((3, 640), 2.5), torch.zeros(2, 640)])
    y, rstd = torch.empty(5, 640, device=DEV), torch.empty(5, device=DEV)
    beta = torch.randn(640, generator=gen(1)).to(DEV)
    a.zs_norm_forward(5, 640, x.to(DEV), y, None, beta, eps=EPS, rstd=rstd)
    assert torch.equal(y, beta.expand(5, 640))
    want = torch.full((5,), 1 / np.sqrt(np.float64(np.float32(EPS))))
    assert torch.allclose(rstd.cpu().double(), want.double(), rtol=3 * ref.U)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_of_non_finite_rows(kind):
    x = torch.randn(8, 1030, generator=gen(2))
    x[1, 5], x[3, 1029], x[6, 700] = float("nan"), float("inf"), float("-inf")
    clean = x.clone()
    clean[[1, 3, 6]] = 0
    out = []
    for v in (x, clean):
        y = torch.empty(8, 1030, dtype=torch.bfloat16, device=DEV)
        a.zs_norm_forward(8, 1030, v.bfloat16().to(DEV), y, kind=kind)
        out.append(y.float().cpu())
    for r in range(8):
        if r in (1, 3, 6):
            assert not torch.isfinite(out[0][r]).all()
        else:
            assert torch.equal(out[0][r], out[1][r])


def test_norm_overflow_and_tiny_values():
    # squares beyond fp32: infinite variance, rstd 0
    y = torch.empty(1, 256, device=DEV)
    a.zs_norm_forward(1, 256, torch.full((1, 256), 1e30, device=DEV), y, kind="rms")
    assert torch.equal(y, torch.zeros_like(y))
    run_norm(4, 300, "layer", "f32", x=torch.randn(4, 300, generator=gen(1)) * 1e-18, present=(False, False))


# ----------------------------------------------------------------- its backward pass

def run_norm_grad(rows, cols, kind, dt, wdt="bf16", gdt="f32", dres=False, accumulate=False, shift=0, gap=0,
                  gamma=True, want=(True, True), seed=0, place=None):
    dtype, gdtype = TD[dt], TD[gdt]
    X = Buf(rows, cols, dtype, shift, gap, activations(rows, cols, seed))
    D = Buf(rows, cols, dtype, 2 * shift, gap, torch.randn(rows, cols, generator=gen(seed + 1)))
    R = Buf(rows, cols, dtype, shift, 2 * gap, torch.randn(rows, cols, generator=gen(seed + 2))) if dres else None
    G = weights(cols, wdt, seed + 3, (gamma, False))[0]
    x64, d64 = X.cpu64(), D.cpu64()
    r64 = R.cpu64() if dres else torch.zeros_like(x64)
    mean = x64.mean(1).float() if kind == "layer" else None
    rstd = ((x64 - (mean.double()[:, None] if mean is not None else 0)).square().mean(1) + EPS).rsqrt().float()
    O = {None: Buf(rows, cols, dtype, shift, gap), "dx=dy": D, "dx=x": X, "dx=dres": R}[place] \
        if place else Buf(rows, cols, dtype, shift, gap)
    grads = [Buf(1, cols, gdtype, shift, 0, torch.randn(1, cols, generator=gen(seed + 4 + i))) if w else None
             for i, w in enumerate(want)]
    old = [g.cpu64()[0] if g and accumulate else torch.zeros(cols, dtype=torch.float64) for g in grads]
    nb = a.zs_norm_workspace_bytes(rows, cols)
    ws = garbage(nb + 256)
    a.zs_norm_backward(rows, cols, D.t, X.t, rstd.to(DEV), O.t, mean=None if mean is None else mean.to(DEV),
                       gamma=G, dres=R.t if R else None, dgamma=grads[0].t[0] if grads[0] else None,
                       dbeta=grads[1].t[0] if grads[1] else None, kind=kind, accumulate=accumulate,
                       workspace=ws if any(want) else None, ws_bytes=nb)
    if rows == 0:
        return grads
    exact = ref.norm_grad(d64, x64, mean.double() if mean is not None else None, rstd.double(), wide(G, cols, 1.0),
                          r64, kind, dtype, gdtype, *old)
    within(O.t, exact["dx"], "dx")
    for name, g in zip(("dgamma", "dbeta"), grads):
        if g:
            within(g.t[0], exact[name], name)
    for b in (X, D, R, O, *grads):
        if b:
            b.check("buffer")
    assert bool((ws[nb:] == 0xFF).all())
    return grads


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_norm_grad_of_every_width(kind, dt):
    for i, cols in enumerate(COLS):
        run_norm_grad(11, cols, kind, dt, seed=i)


@pytest.mark.parametrize("dt,gdt", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("rows,cols", [(1, 4096), (2, 768), (7, 100), (1000, 33), (4097, 768), (9001, 40),
                                       (3001, 600), (1037, 5000), (2100, 1500), (600, 16384)])
def test_norm_grad_of_many_rows(rows, cols, dt, gdt):
    run_norm_grad(rows, cols, "layer", dt, gdt=gdt, dres=True, accumulate=True, seed=rows)
    run_norm_grad(rows, cols, "rms", dt, gdt=gdt, want=(True, False), seed=rows)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt,wdt,gdt", [("bf16", "f32", "f16"), ("f16", "bf16", "bf16"), ("f32", "f16", "f16"),
                                        ("f32", "f32", "bf16"), ("f16", "f16", "f32")])
@pytest.mark.parametrize("shift,gap", [(1, 0), (3, 5), (8, 8)])
def test_norm_grad_at_odd_places(kind, dt, wdt, gdt, shift, gap):
    for cols in (31, 768, 1001, 4100):
        run_norm_grad(37, cols, kind, dt, wdt, gdt, dres=True, accumulate=cols % 2 == 0, shift=shift, gap=gap,
                      seed=cols)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("want", [(True, False), (False, True), (False, False), (True, True)])
def test_norm_grad_of_what_is_wanted(kind, want):
    run_norm_grad(70, 700, kind, "bf16", want=want, gamma=False)
    run_norm_grad(9, 10_000, kind, "bf16", want=want)


@pytest.mark.parametrize("place", ["dx=dy", "dx=x", "dx=dres"])
@pytest.mark.parametrize("rows,cols", [(2500, 100), (2500, 768), (2500, 6000), (400, 768), (90, 5000), (1, 31)])
def test_norm_grad_in_place(place, rows, cols):
    run_norm_grad(rows, cols, "layer", "bf16", dres=True, place=place)


@pytest.mark.parametrize("dt,gdt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,cols", NARROW)
def test_norm_grad_of_narrow_rows(rows, cols, dt, gdt):
    run_norm_grad(rows, cols, "layer", dt, "f32", gdt, dres=True, accumulate=True, gap=cols, seed=rows)
    run_norm_grad(rows, cols, "rms", dt, gdt=gdt, seed=rows, place="dx=x")


@pytest.mark.parametrize("dt,gdt", [("bf16", "f16"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("cols", REMAINDERS)
def test_norm_grad_of_every_remainder(cols, dt, gdt):
    for rows in (9, 1100):
        run_norm_grad(rows, cols, "layer", dt, "f16", gdt, dres=True, accumulate=True, shift=1, gap=1, seed=cols)
        run_norm_grad(rows, cols, "rms", dt, "f32", gdt, gap=2, place="dx=dy", seed=cols)


def test_norm_grad_of_columns_of_one_buffer():
    """dy, x and dx side by side in the same rows, few enough to be read twice."""
    g = gen(4)
    b = torch.randn(300, 3 * 256, generator=g).bfloat16().to(DEV)
    dy, x, dx = b[:, :256], b[:, 256:512], b[:, 512:]
    keep = b[:, :512].clone()
    rstd, dg = torch.rand(300, generator=g).to(DEV), torch.empty(256, device=DEV)
    nb = a.zs_norm_workspace_bytes(300, 256)
    a.zs_norm_backward(300, 256, dy, x, rstd, dx, dgamma=dg, kind="rms", workspace=garbage(nb), ws_bytes=nb)
    zero, one = torch.zeros(256, dtype=torch.float64), torch.ones(256, dtype=torch.float64)
    want = ref.norm_grad(keep[:, :256].cpu().double(), keep[:, 256:].cpu().double(), None, rstd.cpu().double(), one,
                         torch.zeros(300, 256, dtype=torch.float64), "rms", torch.bfloat16, torch.float32, zero, zero)
    within(dx, want["dx"], "dx")
    within(dg, want["dgamma"], "dgamma")
    assert torch.equal(b[:, :512], keep)


def test_norm_grad_of_no_rows():
    g = run_norm_grad(0, 300, "layer", "bf16", gdt="bf16")
    assert all(bool((b.t == 0).all()) for b in g)
    g = run_norm_grad(0, 300, "layer", "bf16", gdt="bf16", accumulate=True)
    assert torch.equal(g[0].t, torch.randn(1, 300, generator=gen(4)).bfloat16().to(DEV))


def test_norm_grad_of_non_finite_rows():
    """They reach their own row of dx and the weights' sums, and no other row."""
    x, dy = (torch.randn(300, 530, generator=gen(s)) for s in (1, 2))
    bad = dy.clone()
    bad[17, 3] = float("inf")
    rstd, mean = torch.ones(300, device=DEV), torch.zeros(300, device=DEV)
    nb = a.zs_norm_workspace_bytes(300, 530)
    out = []
    for d in (dy, bad):
        dx, dg = torch.empty(300, 530, device=DEV), torch.empty(530, device=DEV)
        a.zs_norm_backward(300, 530, d.to(DEV), x.to(DEV), rstd, dx, mean=mean, dgamma=dg,
                           workspace=garbage(nb), ws_bytes=nb)
        out.append((dx.cpu(), dg.cpu()))
    other = torch.arange(300) != 17
    assert torch.equal(out[0][0][other], out[1][0][other]) and not torch.isfinite(out[1][0][17]).all()
    cols = torch.arange(530) != 3
    assert torch.equal(out[0][1][cols], out[1][1][cols]) and not torch.isfinite(out[1][1][3])


@pytest.mark.parametrize("dt,cols", [("bf16", c) for c in (8, 72, 136, 264, 520, 768, 1032, 2056, 4104, 5120, 8200, 9000)]
                         + [("f32", c) for c in (4, 36, 132, 260, 516, 1028, 8196, 9000)] + [("f32", 9001), ("bf16", 71)])
@pytest.mark.parametrize("rows", [3, 1100])
def test_norm_grad_of_huge_equal_values(dt, cols, rows):
    """mean * rstd is beyond fp32 and x - mean is 0: the lanes of a team behind a row's last element see
    the mean, and not the row."""
    x = Buf(rows, cols, TD[dt], values=torch.full((rows, cols), 2.0 ** 110)).t
    dy = Buf(rows, cols, TD[dt], values=torch.randn(rows, cols, generator=gen(cols))).t
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    gamma = weights(cols, "bf16", 5, (True, False))[0]
    a.zs_norm_forward(rows, cols, x, y, gamma, eps=1e-12, mean=mean, rstd=rstd)
    dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    nb = a.zs_norm_workspace_bytes(rows, cols)
    a.zs_norm_backward(rows, cols, dy, x, rstd, dx, mean=mean, gamma=gamma, dgamma=dg, dbeta=db,
                       workspace=garbage(nb), ws_bytes=nb)
    assert bool((mean == 2.0 ** 110).all()) and bool((rstd * 2.0 ** 110 == float("inf")).all())
    zero = torch.zeros(rows, cols, dtype=torch.float64)
    want = ref.norm_grad(dy.cpu().double(), x.cpu().double(), mean.cpu().double(), rstd.cpu().double(),
                         wide(gamma, cols, 1.0), zero, "layer", TD[dt], torch.float32, zero[0], zero[0])
    for got, name in ((dx, "dx"), (dg, "dgamma"), (db, "dbeta")):
        within(got, want[name], name)


@pytest.mark.parametrize("cols", [4, 35, 36, 128, 516, 768, 9000])
def test_norm_grad_of_an_infinite_rstd(cols):
    """Squares that vanish and no eps: h and c2 are +inf, so dx = (1 - inf * inf) * inf, whatever the width."""
    x, one = torch.full((3, cols), 1e-30, device=DEV), torch.ones(3, cols, device=DEV)
    y, dx, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(3, device=DEV)
    a.zs_norm_forward(3, cols, x, y, kind="rms", eps=0.0, rstd=rstd)
    a.zs_norm_backward(3, cols, one, x, rstd, dx, kind="rms")
    assert bool((rstd == float("inf")).all()) and bool((dx == -float("inf")).all())


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_grad_against_differences(kind):
    """Along a direction d: the outputs of two forward passes 2h apart, in fp32.  Each output is off
    by at most the reference's bound, so the difference of the two weighted sums is off by at most
    twice the bounds' weighted sum, over 2h; the cubic term is h^2 / 6 times a third derivative of
    the weighted sum, which for rows of unit scale is below 60 |dy| |d|^3 / rows' scale."""
    rows, cols, h = 40, 768, 2e-2
    g = gen(11)
    x, dy, d = (torch.randn(rows, cols, generator=g) for _ in range(3))
    d /= d.norm(dim=1, keepdim=True)
    gamma, beta = weights(cols, "f32", 12, (True, True))
    kw = dict(kind=kind, eps=EPS)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    y = torch.empty(rows, cols, device=DEV)
    a.zs_norm_forward(rows, cols, x.to(DEV), y, gamma, beta, mean=mean, rstd=rstd, **kw)
    dx, dg, db = torch.empty(rows, cols, device=DEV), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    nb = a.zs_norm_workspace_bytes(rows, cols)
    a.zs_norm_backward(rows, cols, dy.to(DEV), x.to(DEV), rstd, dx, mean=mean, gamma=gamma, dgamma=dg, dbeta=db,
                       kind=kind, workspace=garbage(nb), ws_bytes=nb)

    def weighted(x, gamma, beta):
        out = torch.empty(rows, cols, device=DEV)
        a.zs_norm_forward(rows, cols, x.to(DEV), out, gamma, beta, **kw)
        bound = ref.norm(x.double(), gamma.cpu().double(), beta.cpu().double(), kind, float(np.float32(EPS)),
                         torch.float32)["y"][1]
        return (out.cpu().double() * dy.double()).sum(), (bound * dy.double().abs()).sum()

    dv = torch.randn(cols, generator=g).to(DEV)
    for got, up, down in ((float((dx.cpu().double() * d.double()).sum()), (x + h * d, gamma, beta),
                           (x - h * d, gamma, beta)),
                          (float((dg.double() * dv.double()).sum()), (x, gamma + h * dv, beta), (x, gamma - h * dv, beta)),
                          (float((db.double() * dv.double()).sum()), (x, gamma, beta + h * dv), (x, gamma, beta - h * dv))):
        (u, bu), (v, bv) = weighted(*up), weighted(*down)
        # x + h d itself is rounded: half a step of values below 5, in every term
        moved = 2 * 4 * ref.U * float((dy.abs().double() * (1 + gamma.abs().max().cpu().double())).sum())
        third = h * h / 6 * 60 * float(dy.double().norm(dim=1).sum()) / cols
        assert abs(got - float(u - v) / (2 * h)) <= float(bu + bv + moved) / (2 * h) + third


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows,cols", [(40, 768), (1200, 768), (30, 1001)])
def test_norm_grad_against_close_differences(kind, rows, cols):
    """Row by row, within 2% of the derivative (layer_diff derives by how much); 1200 rows take two launches."""
    x, dy, gamma, beta = layer_diff.inputs(rows, cols, rows + cols)
    G, B = gamma.to(DEV), beta.to(DEV)

    def forward(x, gamma, beta, **kw):
        y = torch.empty(rows, cols, device=DEV)
        a.zs_norm_forward(rows, cols, x.to(DEV), y, gamma.to(DEV), beta.to(DEV), kind=kind, eps=EPS, **kw)
        return y.cpu()

    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    forward(x, G, B, mean=mean, rstd=rstd)
    dx, dg, db = torch.empty(rows, cols, device=DEV), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    nb = a.zs_norm_workspace_bytes(rows, cols)
    a.zs_norm_backward(rows, cols, dy.to(DEV), x.to(DEV), rstd, dx, mean=mean, gamma=G, dgamma=dg, dbeta=db,
                       kind=kind, workspace=garbage(nb), ws_bytes=nb)
    layer_diff.check(forward, x, dy, gamma, beta, kind, float(np.float32(EPS)), dx.cpu(), dg.cpu(), db.cpu())


# ----------------------------------------------------------------- the table

def run_embed(tokens, rows, cols, dt, tdt, ids=None, id_type=torch.int64, scale=1.0, first=0, pos=0, shift=0, gap=0,
              seed=0):
    g = gen(seed)
    if ids is None:
        ids = torch.randint(first - 2, first + rows + 2, (tokens,), generator=g)
    T = Buf(1, rows * cols, TD[tdt], shift, 0, torch.randn(1, rows * cols, generator=g))
    Y = Buf(tokens, cols, TD[dt], shift, gap)
    P = p_ids = None
    row = ids - first
    inside = ((row >= 0) & (row < rows))[:, None]
    want = T.t[0].cpu().float().view(rows, cols)[row.clamp(0, rows - 1)] * torch.tensor(scale, dtype=torch.float32)
    want = torch.where(inside, want, torch.zeros(()))
    if pos:
        P = Buf(1, pos * cols, TD[tdt], 2 * shift, 0, torch.randn(1, pos * cols, generator=g))
        p_ids = torch.randint(-1, pos + 1, (tokens,), generator=g)
        there = ((p_ids >= 0) & (p_ids < pos))[:, None]
        add = P.t[0].cpu().float().view(pos, cols)[p_ids.clamp(0, pos - 1)]
        want = torch.where(there, want + add, want)
    a.zs_embed_forward(tokens, ids.to(id_type).to(DEV), rows, cols, T.t[0], Y.t, scale=scale, first_row=first,
                       pos_ids=None if not pos else p_ids.to(id_type).to(DEV), pos_rows=pos,
                       pos_table=P.t[0] if pos else None)
    assert torch.equal(Y.t.cpu(), want.to(TD[dt]))       # the stated operations have one result
    Y.check("y")


@pytest.mark.parametrize("dt,tdt", [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("bf16", "f32"), ("f16", "bf16"),
                                    ("f32", "f32"), ("f32", "f16"), ("f16", "f32"), ("bf16", "f16")])
def test_embed(dt, tdt):
    for i, (tokens, rows, cols) in enumerate([(1, 1, 1), (5, 3, 7), (64, 100, 64), (33, 50, 515), (300, 70, 768),
                                              (9, 20, 4099), (1500, 17, 8), (2, 5, 20_000)]):
        run_embed(tokens, rows, cols, dt, tdt, seed=i, scale=cols ** 0.5, pos=(i % 3) * 5,
                  id_type=(torch.int64, torch.int32)[i % 2], first=(0, 1000)[i % 2])
        run_embed(tokens, rows, cols, dt, tdt, seed=i, shift=1 + i, gap=i, pos=((i + 1) % 3) * 5, first=7)


@pytest.mark.parametrize("dt,tdt", [("bf16", "f16"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("cols", REMAINDERS)
def test_embed_of_every_remainder(cols, dt, tdt):
    run_embed(40, 30, cols, dt, tdt, seed=cols, pos=20, shift=1, gap=1, scale=3.3)


def test_embed_ids_of_any_value():
    extremes = torch.tensor([0, 1, 49, 50, -1, 2**31 - 1, -2**31, 2**31, 2**32, 2**32 + 3, 2**63 - 1, -2**63, 7])
    run_embed(13, 50, 100, "f32", "f32", ids=extremes)
    run_embed(13, 50, 100, "f32", "f32", ids=extremes.clamp(-2**31, 2**31 - 1), id_type=torch.int32)
    for id_type, top in ((torch.int64, 2**63 - 1), (torch.int32, 2**31 - 1)):
        n = torch.tensor([top, top - 1, top - 49, top - 50, 0])
        run_embed(5, 50, 100, "f32", "f32", ids=n, first=top - 49, id_type=id_type)


def test_embed_of_a_missing_row_is_plus_zero():
    y = torch.full((1, 32), -1.0, dtype=torch.bfloat16, device=DEV)
    t = torch.full((4, 32), float("nan"), dtype=torch.bfloat16, device=DEV)
    a.zs_embed_forward(1, torch.tensor([-1], device=DEV), 4, 32, t, y, scale=-2.0)
    assert bool((y.view(torch.int16) == 0).all())


def token_ids(tokens, rows, kind, seed):
    g = gen(seed)
    if kind == "zipf":
        return ((torch.rand(tokens, generator=g, dtype=torch.float64) * np.log(rows + 1)).exp() - 1).long()
    if kind == "one":
        return torch.full((tokens,), rows // 2)
    if kind == "each":
        return torch.randperm(max(tokens, rows), generator=g)[:tokens] % rows
    if kind == "runs":      # runs that end on and next to the chunks' ends
        return (torch.arange(tokens) // 32 + (torch.arange(tokens) % 97 == 0).long()) % rows
    if kind == "none":
        return torch.full((tokens,), -1)
    return torch.randint(-rows, 2 * rows, (tokens,), generator=g)      # "part": most are no row here


def run_embed_grad(tokens, rows, cols, kind, dt="bf16", gdt="f32", accumulate=False, scale=1.0, first=0,
                   id_type=torch.int64, shift=0, gap=0, seed=0, whole_numbers=False):
    g = gen(seed + 1)
    row = token_ids(tokens, rows, kind, seed)
    row = torch.where((row >= 0) & (row < rows), row, torch.tensor(-1))
    dy = torch.randint(-4, 5, (tokens, cols), generator=g).float() if whole_numbers \
        else torch.randn(tokens, cols, generator=g)
    D = Buf(tokens, cols, TD[dt], shift, gap, dy)
    G = Buf(1, rows * cols, TD[gdt], shift, 0,
            torch.randint(-9, 10, (1, rows * cols), generator=g).float() if whole_numbers
            else torch.randn(1, rows * cols, generator=g))
    old = G.t[0].cpu().double().view(rows, cols) if accumulate else torch.zeros(rows, cols, dtype=torch.float64)
    nb = a.zs_embed_workspace_bytes(tokens, rows, cols)
    ws = garbage(nb + 256)
    ids = torch.where(row >= 0, row + first, row).to(id_type).to(DEV)
    before = G.t[0].clone()
    a.zs_embed_backward(tokens, ids, rows, cols, D.t, G.t[0], ws, nb, scale=scale, first_row=first,
                        accumulate=accumulate)
    value, bound, count = ref.embed_grad(D.cpu64(), row, rows, float(np.float32(scale)), old, TD[gdt])
    got = G.t[0].view(rows, cols)
    if whole_numbers:       # sums below 2^24: exact in any order
        assert torch.equal(got.cpu().double(), value)
    else:
        within(got, (value, bound), kind)
    if accumulate:          # rows that no token names stay as they were
        idle = (count == 0).to(DEV)
        raw = torch.int32 if gdt == "f32" else torch.int16
        assert torch.equal(got.view(raw)[idle], before.view(rows, cols).view(raw)[idle])
    D.check("dy")
    G.check("grad")
    assert bool((ws[nb:] == 0xFF).all())


KINDS = ["zipf", "one", "each", "runs", "none", "part"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_of_whole_numbers(kind, accumulate):
    for i, (tokens, rows, cols) in enumerate([(1, 1, 1), (2, 3, 9), (31, 5, 40), (32, 5, 40), (33, 5, 40),
                                              (64, 700, 64), (65, 7, 33), (1000, 300, 100), (1023, 2000, 520),
                                              (1024, 2000, 513), (1025, 1023, 16), (2049, 1024, 24),
                                              (4096, 1025, 8), (5000, 5000, 12)]):
        run_embed_grad(tokens, rows, cols, kind, accumulate=accumulate, whole_numbers=True, seed=i,
                       first=(0, 5000)[i % 2], id_type=(torch.int64, torch.int32)[i % 2])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [16_384, 16_385, 32_768, 32_769, 40_000, 65_536, 131_072, 131_073, 600_000])
def test_embed_grad_of_long_batches(kind, tokens):
    run_embed_grad(tokens, 3001, 24, kind, whole_numbers=True, seed=tokens, accumulate=tokens % 2 == 0)
    run_embed_grad(tokens, 70_000, 5, kind, whole_numbers=True, seed=tokens, accumulate=tokens % 2 == 1)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gdt", ["bf16", "f16", "f32"])
def test_embed_grad(dt, gdt):
    for i, (tokens, rows, cols, kind) in enumerate([(500, 90, 515, "zipf"), (77, 1000, 4099, "each"),
                                                    (2000, 40, 768, "zipf"), (300, 3, 64, "one"),
                                                    (901, 333, 31, "part")]):
        run_embed_grad(tokens, rows, cols, kind, dt, gdt, accumulate=i % 2 == 0, scale=cols ** 0.5, seed=i)
        run_embed_grad(tokens, rows, cols, kind, dt, gdt, accumulate=i % 2 == 1, scale=-0.3, seed=i, shift=1 + i,
                       gap=i + 1)


@pytest.mark.parametrize("dt,gdt", [("bf16", "f16"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("cols", REMAINDERS)
def test_embed_grad_of_every_remainder(cols, dt, gdt):
    """Short rows, long ones, and rows that the gradient already holds."""
    for kind in ("each", "zipf"):
        run_embed_grad(300, 20, cols, kind, dt, gdt, accumulate=kind == "zipf", seed=cols, shift=1, gap=1)
        run_embed_grad(300, 20, cols, kind, dt, gdt, accumulate=kind == "each", seed=cols)


@pytest.mark.parametrize("kind", KINDS)
def test_embed_grad_of_small_tables(kind):
    """No more rows than buckets of the sort, with few and with many tokens each."""
    for i, (tokens, rows) in enumerate([(300, 1), (3000, 1), (3000, 5), (16_384, 64), (16_384, 65), (900, 64)]):
        run_embed_grad(tokens, rows, 16, kind, whole_numbers=True, seed=i, accumulate=i % 2 == 0)


@pytest.mark.parametrize("kind", ["zipf", "one", "part"])
def test_embed_grad_of_a_large_table(kind):
    """Cleared by small workgroups beside the sort.  Whole numbers: any order gives the same sums."""
    rows, cols, tokens = 140_001, 1000, 16_000
    row = token_ids(tokens, rows, kind, 5).to(DEV)
    dy = torch.randint(-4, 5, (tokens, cols), generator=gen(6)).bfloat16().to(DEV)
    G = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    nb = a.zs_embed_workspace_bytes(tokens, rows, cols)
    a.zs_embed_backward(tokens, row, rows, cols, dy, G, garbage(nb), nb)
    inside = (row >= 0) & (row < rows)
    want = torch.zeros(rows, cols, device=DEV).index_add_(0, row[inside], dy[inside].float())
    assert torch.equal(G, want.bfloat16())


def test_embed_grad_of_many_rows():
    """Rows whose number takes two and three digits of the sort, and the last row."""
    for rows in (1 << 10, (1 << 20) - 1, 1 << 20, (1 << 20) + 5, 5_000_000):
        ids = torch.tensor([rows - 1, 0, rows // 2, rows - 1, rows - 2, -1, rows, 0])
        dy = torch.randint(-4, 5, (8, 4), generator=gen(rows)).float()
        for n in (8, 8 * 5000, 8 * 20_000):        # in one launch, and in several
            G = torch.full((rows, 4), 7.0, device=DEV)
            nb = a.zs_embed_workspace_bytes(n, rows, 4)
            a.zs_embed_backward(n, ids.repeat(n // 8).to(DEV), rows, 4, dy.repeat(n // 8, 1).to(DEV), G, garbage(nb), nb)
            want = torch.zeros(rows, 4).index_add_(0, ids[[0, 1, 2, 3, 4, 7]], dy[[0, 1, 2, 3, 4, 7]] * (n // 8))
            assert torch.equal(G.cpu(), want)


def test_embed_grad_of_no_tokens():
    G = torch.full((50, 33), 3.0, dtype=torch.bfloat16, device=DEV)
    a.zs_embed_backward(0, None, 50, 33, None, G, accumulate=True, dtype="bf16", id_dtype="i64")
    assert bool((G == 3).all())
    a.zs_embed_backward(0, None, 50, 33, None, G, dtype="bf16", id_dtype="i64")
    assert bool((G.view(torch.int16) == 0).all())


def test_embed_grad_does_not_read_what_has_no_row():
    """dy of padding may hold anything."""
    dy = torch.full((400, 80), float("nan"))
    ids = torch.full((400,), -1)
    ids[::10] = torch.arange(40) % 7
    dy[::10] = 1.0
    nb = a.zs_embed_workspace_bytes(400, 9, 80)
    G = torch.empty(9, 80, device=DEV)
    a.zs_embed_backward(400, ids.to(DEV), 9, 80, dy.to(DEV), G, garbage(nb), nb)
    assert torch.equal(G.cpu(), torch.bincount(ids[::10], minlength=9).float()[:, None].expand(9, 80))


# ----------------------------------------------------------------- sizes, streams, graphs

def test_offsets_beyond_32_bits():
    """Rows and tables that end behind 2^32 elements."""
    stride = (1 << 31) + 64
    base = torch.zeros(2 * stride + 4096, dtype=torch.bfloat16, device=DEV)
    x = base.as_strided((3, 1000), (stride, 1))
    x.copy_(torch.randn(3, 1000, generator=gen(1)).to(DEV))
    y = base.as_strided((3, 1000), (stride, 1), 2048)
    a.zs_norm_forward(3, 1000, x, y, kind="rms", eps=EPS)
    want = ref.norm(x.cpu().double(), torch.ones(1000).double(), torch.zeros(1000).double(), "rms",
                    float(np.float32(EPS)), torch.bfloat16)
    within(y, want["y"], "y")
    dy = base.as_strided((3, 1000), (stride, 1), 2048)
    G = torch.zeros(5, 1000, device=DEV)
    nb = a.zs_embed_workspace_bytes(3, 5, 1000)
    a.zs_embed_backward(3, torch.tensor([4, 1, 4], device=DEV), 5, 1000, dy, G, garbage(nb), nb)
    e = torch.zeros(5, 1000).index_add_(0, torch.tensor([4, 1, 4]), dy.float().cpu())
    assert torch.equal(G.cpu(), e)
    del base, x, y, dy
    rows, cols = (1 << 22) + 3, 1032
    table = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    ids = torch.tensor([rows - 1, 0, rows - 2, rows - 1], device=DEV)
    src = torch.randint(-8, 9, (4, cols), generator=gen(2)).bfloat16().to(DEV)
    nb = a.zs_embed_workspace_bytes(4, rows, cols)
    a.zs_embed_backward(4, ids, rows, cols, src, table, garbage(nb), nb, accumulate=True)
    assert torch.equal(table[rows - 1], src[0] + src[3]) and torch.equal(table[rows - 2], src[2])
    out = torch.empty(4, cols, dtype=torch.bfloat16, device=DEV)
    a.zs_embed_forward(4, ids, rows, cols, table, out)
    assert torch.equal(out, table[ids])
    table.fill_(1.0)
    a.zs_embed_backward(4, ids, rows, cols, src, table, garbage(nb), nb)
    assert torch.equal(table[rows - 1], src[0] + src[3]) and torch.equal(table[0], src[1])
    assert float(table[1:rows - 2].abs().max()) == 0.0


# ----------------------------------------------------------------- the kernels that large inputs take

def many_tokens(tokens, rows, cols, dt, gdt, accumulate, seed, gap=0):
    """Whole numbers, so that any order gives the same sums, compared on the device.  Half of the tokens name few
    rows (whose tokens are summed in parts), a quarter name rows evenly, and the others none."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    row = torch.randint(0, rows, (tokens,), generator=g, device=DEV)
    kind = torch.rand(tokens, generator=g, device=DEV)
    row = torch.where(kind < 0.5, row % 40, torch.where(kind < 0.75, row, torch.full_like(row, -1)))
    dy = torch.randint(-4, 5, (tokens, cols + gap), generator=g, device=DEV, dtype=torch.int8).to(TD[dt])[:, :cols]
    old = torch.randint(-9, 10, (rows, cols), generator=g, device=DEV, dtype=torch.int8)
    grad = Buf(1, rows * cols, TD[gdt], 1, 0, old.view(1, -1))
    nb = a.zs_embed_workspace_bytes(tokens, rows, cols)
    ws = garbage(nb + 256)
    a.zs_embed_backward(tokens, row, rows, cols, dy, grad.t[0], ws, nb, accumulate=accumulate)
    want = old.float() if accumulate else torch.zeros(rows, cols, device=DEV)
    inside = row >= 0
    want.index_add_(0, row[inside], dy[inside].float())
    assert torch.equal(grad.t[0].view(rows, cols), want.to(TD[gdt]))
    grad.check("grad")
    assert bool((ws[nb:] == 0xFF).all())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("gdt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_embed_grad_of_many_tokens(dt, gdt, accumulate):
    """More than 2^23 elements of dy, in whole packs and in broken ones, sorted in one launch and in several."""
    for i, (tokens, cols) in enumerate([(8400, 1000), (8200, 1025), (16_500, 515), (33_000, 256)]):
        many_tokens(tokens, 3001, cols, dt, gdt, accumulate, seed=i, gap=i % 2)


@pytest.mark.parametrize("cols", [1000, 1001, 1004, 4096])
@pytest.mark.parametrize("gdt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_embed_grad_of_more_than_the_cache_keeps(dt, gdt, cols):
    """More than 64 MiB of dy, added to a gradient: read past the cache."""
    tokens = (1 << 26) // (cols * (4 if dt == "f32" else 2)) + 1
    many_tokens(tokens, 700, cols, dt, gdt, True, seed=cols)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", [512, 4096, 16384])
def test_norm_of_more_than_the_cache_keeps(kind, residual, dt, cols):
    """More than 192 MiB read and written: read past the cache.  Against the 64-bit reference, on the device."""
    each = cols * (4 if dt == "f32" else 2) * (4 if residual else 2)
    rows = (192 << 20) // each + 1
    g = torch.Generator(device=DEV).manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, device=DEV) * (0.2 + 2 * torch.rand(rows, 1, generator=g, device=DEV))
    x[:, :: 97] *= 15
    x = x.to(TD[dt])
    r = torch.randn(rows, cols, generator=g, device=DEV).to(TD[dt]) if residual else None
    total = torch.empty_like(x) if residual else None
    y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    mean = torch.empty(rows, device=DEV) if kind == "layer" else None
    gamma, beta = weights(cols, "f32", 3, (True, True))
    a.zs_norm_forward(rows, cols, x, y, gamma, beta, kind=kind, eps=EPS, residual=r, total=total, mean=mean, rstd=rstd)
    t = x
    if residual:
        t = (x.float() + r.float()).to(TD[dt])
        assert torch.equal(total, t)
    for i in range(0, rows, 4096):
        at = slice(i, i + 4096)
        with torch.device(DEV):
            want = ref.norm(t[at].double(), gamma.double(), beta.double(), kind, float(np.float32(EPS)), TD[dt])
        for got, name in ((y, "y"), (rstd, "rstd"), (mean, "mean")):
            if got is not None:
                value, bound = want[name]
                assert bool(((got[at].double() - value).abs() <= bound).all()), name


class Layer:
    """One batch through the lookup, a norm and their backward passes, all buffers kept."""

    def __init__(self, seed, tokens=700, rows=400, cols=768):
        self.n, self.rows, self.cols = tokens, rows, cols
        t = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        self.ids = torch.empty(tokens, dtype=torch.int64, device=DEV)
        self.table, self.dtable = t(rows, cols), t(rows, cols)
        self.gamma, self.dgamma = t(cols), torch.empty(cols, device=DEV)
        self.beta, self.dbeta = t(cols), torch.empty(cols, device=DEV)
        self.x, self.y, self.dy, self.dx = (t(tokens, cols) for _ in range(4))
        self.mean, self.rstd = torch.empty(tokens, device=DEV), torch.empty(tokens, device=DEV)
        self.nb = a.zs_norm_workspace_bytes(tokens, cols), a.zs_embed_workspace_bytes(tokens, rows, cols)
        self.ws = garbage(max(self.nb))      # one after the other: they may share it
        self.fill(seed)

    def fill(self, seed):
        g = gen(seed)
        self.ids.copy_(torch.randint(-1, self.rows, (self.n,), generator=g))
        for x in (self.table, self.gamma, self.beta, self.dy):
            x.copy_(torch.randn(x.shape, generator=g))

    def run(self, stream=None):
        a.zs_embed_forward(self.n, self.ids, self.rows, self.cols, self.table, self.x, scale=2.0, stream=stream)
        a.zs_norm_forward(self.n, self.cols, self.x, self.y, self.gamma, self.beta, mean=self.mean, rstd=self.rstd,
                          stream=stream)
        a.zs_norm_backward(self.n, self.cols, self.dy, self.x, self.rstd, self.dx, mean=self.mean, gamma=self.gamma,
                           dgamma=self.dgamma, dbeta=self.dbeta, workspace=self.ws, ws_bytes=self.nb[0],
                           stream=stream)
        a.zs_embed_backward(self.n, self.ids, self.rows, self.cols, self.dx, self.dtable, self.ws, self.nb[1],
                            scale=2.0, stream=stream)

    def outputs(self):
        return [x.clone() for x in (self.x, self.y, self.mean, self.rstd, self.dx, self.dgamma, self.dbeta,
                                    self.dtable)]


def equal(xs, ys):
    return all(torch.equal(x.view(torch.int32 if x.element_size() == 4 else torch.int16),
                           y.view(torch.int32 if y.element_size() == 4 else torch.int16)) for x, y in zip(xs, ys))


@pytest.mark.parametrize("tokens,rows,cols", [(700, 400, 768), (40_000, 3000, 64), (3000, 100, 4096)])
def test_the_same_bits_every_time(tokens, rows, cols):
    L = Layer(1, tokens, rows, cols)
    L.run()
    first = L.outputs()
    for _ in range(5):
        L.ws.fill_(0xFF)
        L.run()
        assert equal(first, L.outputs())


def test_two_streams_at_once():
    layers = [Layer(s, 5000, 3000, 512) for s in (1, 2)]
    for L in layers:
        L.run()
    torch.cuda.synchronize()
    want = [L.outputs() for L in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for L in layers:
        L.ws.fill_(0xFF)
        for x in (L.x, L.y, L.dx, L.dgamma, L.dbeta, L.dtable):
            x.fill_(0)
    torch.cuda.synchronize()
    for _ in range(5):
        for L, s in zip(layers, streams):
            L.run(s)
    torch.cuda.synchronize()
    for L, w in zip(layers, want):
        assert equal(w, L.outputs())


@pytest.mark.parametrize("tokens", [700, 40_000])
def test_captured_and_replayed(tokens):
    """New inputs in the captured buffers, other work between the replays."""
    L = Layer(1, tokens, 900, 256)
    L.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        L.run(torch.cuda.current_stream())
    E = Layer(1, tokens, 900, 256)
    for seed in (3, 4, 5, 6):
        L.fill(seed)
        E.fill(seed)
        graph.replay()
        E.run()
        torch.cuda.synchronize()
        assert equal(E.outputs(), L.outputs())


# ----------------------------------------------------------------- the operators together

@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_training_steps_of_a_small_model(kind):
    """Tokens and positions through two residual blocks and a tied output projection, the gradients straight into
    the buffers that the AdamW step reads, two micro batches added up; against autograd in 64 bits.  In fp32: a
    pass is some 40 operations deep with sums of at most 400 terms, so the gradients are held to
    40 * 400 * U of their norm."""
    V, P, D, S, B = 300, 16, 96, 16, 6
    T = S * B
    g = gen(21)
    names = ["wte", "wpe", "g1", "b1", "m1", "g2", "b2", "m2", "gf", "bf"]
    shapes = [(V, D), (P, D), (D,), (D,), (D, D), (D,), (D,), (D, D), (D,), (D,)]
    lens = [int(np.prod(s)) for s in shapes]
    offs = np.cumsum([0] + lens)
    flat = lambda: torch.zeros(offs[-1], device=DEV)  # noqa: E731
    w, grad = flat(), flat()
    cut = lambda x: {n: x[o:o + k].view(s) for n, o, k, s in zip(names, offs, lens, shapes)}  # noqa: E731
    p, d = cut(w), cut(grad)
    for n, x in p.items():
        x.copy_(torch.randn(x.shape, generator=g) * (0.1 if x.dim() == 2 else 0.2) + (1.0 if n[0] == "g" else 0.0))
    m, v = flat(), flat()
    nb = aw.zs_adamw_workspace_bytes(lens, 1)
    table_ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    table = aw.zs_adamw_upload([dict(len=k, grads=[grad.data_ptr() + 4 * o], w=w.data_ptr() + 4 * o,
                                     m=m.data_ptr() + 4 * o, v=v.data_ptr() + 4 * o)
                                for o, k in zip(offs[:-1].tolist(), lens)], 1, "f32", None, 32, table_ws, nb)
    sumsq = torch.zeros((), dtype=torch.float64, device=DEV)
    nbytes = max(a.zs_norm_workspace_bytes(T, D), a.zs_embed_workspace_bytes(T, V, D))
    ws = garbage(nbytes)
    pos = (torch.arange(T) % S).to(DEV)
    act = lambda: torch.empty(T, D, device=DEV)  # noqa: E731
    layer = kind == "layer"

    def norm(i, x, residual=None):
        y, total, mean, rstd = act(), act(), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        a.zs_norm_forward(T, D, x, y, p["g" + i], p["b" + i], kind=kind, residual=residual,
                          total=total if residual is not None else None, mean=mean, rstd=rstd)
        return y, (total if residual is not None else x), mean, rstd

    def norm_back(i, dy, saved, dres, add):
        dx = act()
        a.zs_norm_backward(T, D, dy, saved[1], saved[3], dx, mean=saved[2] if layer else None, gamma=p["g" + i],
                           dres=dres, dgamma=d["g" + i], dbeta=d["b" + i], kind=kind, accumulate=add, workspace=ws,
                           ws_bytes=nbytes)
        return dx

    def micro(ids, target, add):
        x0 = act()
        a.zs_embed_forward(T, ids, V, D, p["wte"], x0, scale=D ** 0.5, pos_ids=pos, pos_rows=P, pos_table=p["wpe"])
        n1 = norm("1", x0)
        f1 = n1[0] @ p["m1"]
        n2 = norm("2", f1, x0)
        f2 = n2[0] @ p["m2"]
        nf = norm("f", f2, n2[1])
        logits = nf[0] @ p["wte"].t()
        dlog = (torch.softmax(logits, 1) - torch.nn.functional.one_hot(target, V)) / (2 * T)
        into = (lambda n, x: d[n].add_(x)) if add else (lambda n, x: d[n].copy_(x))
        into("wte", dlog.t() @ nf[0])
        dt = norm_back("f", dlog @ p["wte"], nf, None, add)
        into("m2", n2[0].t() @ dt)
        dt = norm_back("2", dt @ p["m2"].t(), n2, dt, add)
        into("m1", n1[0].t() @ dt)
        dt = norm_back("1", dt @ p["m1"].t(), n1, dt, add)
        a.zs_embed_backward(T, ids, V, D, dt, d["wte"], ws, nbytes, scale=D ** 0.5, accumulate=True)
        a.zs_embed_backward(T, pos, P, D, dt, d["wpe"], ws, nbytes, accumulate=add)

    def loss64(q, ids, target):
        def nrm(i, x):
            mu = x.mean(1, keepdim=True) if layer else 0.0
            return (x - mu) / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + EPS) * q["g" + i] + q["b" + i]

        x = q["wte"][ids] * D ** 0.5 + q["wpe"][pos.cpu()]
        x = x + nrm("1", x) @ q["m1"]
        x = x + nrm("2", x) @ q["m2"]
        return torch.nn.functional.cross_entropy(nrm("f", x) @ q["wte"].t(), target, reduction="sum") / (2 * T)

    for step in (1, 2, 3):
        q = {n: x.detach().cpu().double().requires_grad_() for n, x in p.items()}
        for k in (0, 1):
            ids = torch.randint(0, V, (T,), generator=g)
            ids[: T // 3] = 7
            target = torch.randint(0, V, (T,), generator=g)
            micro(ids.to(DEV), target.to(DEV), k == 1)
            loss64(q, ids, target).backward()
        for n in names:
            far = float((d[n].cpu().double() - q[n].grad).norm() / q[n].grad.norm())
            assert far <= 40 * 400 * ref.U, (n, far)
        before = w.clone()
        aw.zs_grad_sumsq_multi(table, sumsq)
        want = sum(float(x.grad.square().sum()) for x in q.values())
        assert abs(float(sumsq) - want) <= 1e-2 * want
        aw.zs_adamw_step_multi(table, aw.hparams(1e-2, 0.9, 0.95, 1e-8, step, max_norm=1.0), sumsq)
        assert bool((w != before).any()) and bool(torch.isfinite(w).all())
