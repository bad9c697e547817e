"""The AdamW operators on the GPU against the numpy references of adamw_ref: bit
for bit with the stated fp32 sequence, and within the bounds that adamw_ref
derives of the definition in 64 bits."""

import math

import numpy as np
import pytest
import torch

import adamw_ref as ref
from adam_zs_shard_amd import zsadamw as a
from adam_zs_shard_amd import zshard as z
from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
TD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
GAP = 40  # elements between two tensors' buffers, which nothing may write
CANARY = {4: 0x5A5A5A5A, 2: 0x5A5A, 1: 0x5A}
LR, B1, B2, EPS = 3e-4, 0.9, 0.95, 1e-8


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    torch.cuda.synchronize()


def bits_of(x):
    x = x.detach().contiguous().cpu()
    return x.view({4: torch.int32, 2: torch.int16, 1: torch.uint8, 8: torch.int64}[x.element_size()]
                  ).numpy()


def same(got, want, what):
    g, w = bits_of(got), np.ascontiguousarray(want).view({4: np.int32, 2: np.int16, 1: np.uint8}[
        want.dtype.itemsize])
    if want.dtype.kind == "f":
        nan = np.isnan(want)
        assert np.array_equal(nan, np.isnan(got.detach().float().cpu().numpy())), what
        g, w = g[~nan], w[~nan]
    assert g.shape == w.shape, what
    differ = int((g != w).sum())
    assert differ == 0, f"{what}: {differ} of {w.size} differ in bits"


class Buffers:
    """Many tensors in one allocation per kind, GAP canaries between them, the
    first one `shift` elements in."""

    def __init__(self, lens, dtype, shift):
        self.lens, self.dtype = lens, dtype
        size = torch.empty(0, dtype=dtype).element_size()
        self.offs, at = [], GAP
        for n in lens:
            # shift None: every tensor on a 128-byte line
            at = -(-at // 256) * 256 if shift is None else at + shift * (not self.offs)
            self.offs.append(at)
            at += n + GAP
        raw = {4: torch.int32, 2: torch.int16, 1: torch.uint8}[size]
        self.flat = torch.full((at,), CANARY[size], dtype=raw, device=DEV).view(dtype)
        self.canary = torch.ones(at, dtype=torch.bool, device=DEV)
        for n, o in zip(lens, self.offs):
            self.canary[o:o + n] = False
        self.raw, self.size = raw, size

    def __getitem__(self, i):
        return self.flat[self.offs[i]:self.offs[i] + self.lens[i]]

    def fill(self, arrays):
        for i, x in enumerate(arrays):
            self[i].copy_(x if isinstance(x, torch.Tensor) else torch.from_numpy(x))
        return self

    def check(self, what):
        assert bool((self.flat.view(self.raw)[self.canary] == CANARY[self.size]).all()), \
            f"{what}: written outside its tensors"


class Model:
    def __init__(self, lens, p=1, grad="bf16", param="bf16", bits=32, shift=0, seed=0, states=True,
                 mean=False, gscale=1e-3):
        self.lens, self.p, self.grad, self.param, self.bits = lens, p, grad, param, bits
        r = self.rng = np.random.default_rng(seed)
        nb = [-(-n // 256) for n in lens]
        self.decay = [0.1 if n > 300 else 0.0 for n in lens]
        self.lr_scale = [[1.0, 0.5, 2.0][i % 3] for i in range(len(lens))]
        self.index = [int(x) for x in r.integers(0, 1 << 40, len(lens))]
        self.gscale = gscale
        self.g = [Buffers(lens, TD[grad], shift) for _ in range(p)]
        self.draw()
        w = [r.standard_normal(n).astype(np.float32) * np.float32(0.02) for n in lens]
        m = [r.standard_normal(n).astype(np.float32) * np.float32(3e-4) for n in lens]
        v = [(np.abs(r.standard_normal(n)).astype(np.float32) + np.float32(0.1)) ** 2 *
             np.float32(1e-6) for n in lens]
        if not states:
            m, v = [np.zeros_like(x) for x in m], [np.zeros_like(x) for x in v]
        self.w = Buffers(lens, torch.float32, shift).fill(w)
        self.pb = Buffers(lens, TD[param], shift) if param else None
        if bits == 8:
            cm, cv = [ref.encode(x, "m") for x in m], [ref.encode(x, "v") for x in v]
            self.m = Buffers(lens, torch.uint8, shift).fill([c for c, _ in cm])
            self.v = Buffers(lens, torch.uint8, shift).fill([c for c, _ in cv])
            self.ms = Buffers(nb, torch.float32, shift).fill([s for _, s in cm])
            self.vs = Buffers(nb, torch.float32, shift).fill([s for _, s in cv])
        else:
            self.m = Buffers(lens, torch.float32, shift).fill(m)
            self.v = Buffers(lens, torch.float32, shift).fill(v)
        self.mean = Buffers(lens, torch.float32, shift) if mean else None
        self.table = self.upload()

    def draw(self):
        """New gradients, some of them zero."""
        for b in self.g:
            xs = []
            for n in self.lens:
                x = self.rng.standard_normal(n).astype(np.float32) * np.float32(self.gscale)
                x[self.rng.random(n) < 0.05] = 0
                xs.append(x)
            b.fill(xs)

    def pieces(self):
        out = []
        for i, n in enumerate(self.lens):
            q = dict(len=n, grads=[b[i] for b in self.g], w=self.w[i], m=self.m[i], v=self.v[i],
                     weight_decay=self.decay[i], lr_scale=self.lr_scale[i], index=self.index[i])
            if self.pb:
                q["param"] = self.pb[i]
            if self.bits == 8:
                q.update(m_scale=self.ms[i], v_scale=self.vs[i])
            if self.mean:
                q["g_mean"] = self.mean[i]
            out.append(q)
        return out

    def upload(self):
        nb = a.zs_adamw_workspace_bytes(self.lens, self.p)
        self.ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
        return a.zs_adamw_upload(self.pieces(), self.p, self.grad, self.param, self.bits, self.ws, nb)

    def host(self, i):
        d = dict(g=[b[i].float().cpu().numpy() for b in self.g], w=self.w[i].cpu().numpy().copy())
        for k in "mv":
            x = getattr(self, k)[i].cpu().numpy().copy()
            if self.bits == 8:
                d["c" + k], d["s" + k] = x, getattr(self, k + "s")[i].cpu().numpy().copy()
                x = ref.decode(x, d["s" + k], k)
            d[k] = x
        return d

    def all(self):
        bufs = [self.w, self.m, self.v] + ([self.pb] if self.pb else [])
        return bufs + ([self.ms, self.vs] if self.bits == 8 else [])

    def step_and_check(self, step, *, grad_scale=1.0, sumsq=None, max_norm=0.0, rounding="nearest",
                       seed=0, bounds=True, run=None):
        before = [self.host(i) for i in range(len(self.lens))]
        hp = a.hparams(LR, B1, B2, EPS, step, grad_scale=grad_scale, max_norm=max_norm,
                       rounding=rounding, seed=seed)
        dev = None if sumsq is None else torch.tensor(sumsq, dtype=torch.float64, device=DEV)
        (run or a.zs_adamw_step_multi)(self.table, hp, dev)
        gs, _ = ref.scale_of(grad_scale, sumsq, max_norm)
        for i, (n, d) in enumerate(zip(self.lens, before)):
            h = dict(lr=LR * self.lr_scale[i], decay=self.decay[i], beta1=B1, beta2=B2, eps=EPS,
                     step=step, gs=gs)
            w, m, v, *off = ref.step32(ref.mean32(d["g"]), d["w"], d["m"], d["v"], h, self.bits)
            what = f"tensor {i} of {n}"
            got = self.w[i].cpu().numpy()
            if self.bits == 32:
                same(self.w[i], w, what + " w")
            else:
                fine = np.isfinite(w)
                assert np.array_equal(fine, np.isfinite(got)), what
                far = np.abs(got[fine] - w[fine].astype(np.float64))
                assert np.all(far <= off[0][fine]), f"{what} w: {float((far / off[0][fine]).max())}"
            if self.pb:  # a NaN is a NaN, whatever its bits
                fine = ~np.isnan(w)
                assert np.array_equal(fine, ~np.isnan(self.pb[i].float().cpu().numpy()))
                same(self.pb[i][torch.from_numpy(fine).to(DEV)],
                     torch.from_numpy(got[fine]).to(TD[self.param]).view(torch.int16).numpy(),
                     what + " param")
            if self.bits == 32:
                same(self.m[i], m, what + " m")
                same(self.v[i], v, what + " v")
            else:
                lo = hi = None
                if rounding == "stochastic":
                    lo, hi = ref.halves_for(n, self.index[i], step, seed)
                for k, x, r in (("m", m, lo), ("v", v, hi)):
                    codes, scales = ref.encode(x, k, r)
                    same(getattr(self, k)[i], codes, what + f" {k} codes")
                    same(getattr(self, k + "s")[i], scales, what + f" {k} scales")
            if bounds:
                w64, m64, v64, bw, bm, bv = ref.step64(d["g"], d["w"], d["m"], d["v"], h, self.bits)
                assert np.all(np.abs(got - w64) <= bw)
                if self.bits == 32:
                    assert np.all(np.abs(self.m[i].cpu().numpy() - m64) <= bm)
                    assert np.all(np.abs(self.v[i].cpu().numpy() - v64) <= bv)
        for b in self.all() + self.g:
            b.check("buffer")


ODD = [1, 2, 3, 255, 256, 257, 1000, 2047, 2048, 2049, 5, 8192, 8195, 30011]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad,param,p,shift", [
    ("bf16", "bf16", 1, 0), ("f16", "f16", 1, 1), ("f32", "bf16", 1, 0), ("f32", None, 3, 3),
    ("bf16", "f16", 2, 8), ("bf16", None, 5, 2), ("f16", "bf16", 8, 0), ("f16", "f16", 7, 13)])
def test_step_of_odd_tensors(bits, grad, param, p, shift):
    M = Model(ODD, p, grad, param, bits, shift, seed=10 + p)
    M.step_and_check(1)
    M.draw()
    M.step_and_check(1000, grad_scale=0.25)


@pytest.mark.parametrize("bits,rounding", [(32, "nearest"), (8, "nearest"), (8, "stochastic")])
@pytest.mark.parametrize("p,shift", [(1, 0), (1, None), (4, 0), (4, None), (17, 1)])
def test_step_of_large_tensors(bits, rounding, p, shift):
    # enough for the larger workgroups, pieces that end inside one
    M = Model([3_000_001, 513, 1_300_000, 77], p, "bf16", "bf16", bits, shift, seed=20)
    assert M.table.on_lines == (shift is None) and M.table.chunk_elems > 2048
    M.step_and_check(17, rounding=rounding, seed=(7 << 32) + 5)


@pytest.mark.parametrize("bits,rounding", [(32, "nearest"), (8, "nearest"), (8, "stochastic")])
@pytest.mark.parametrize("p", [1, 3])
def test_step_of_odd_tensors_on_lines(bits, rounding, p):
    M = Model(ODD, p, "f16", "bf16", bits, None, seed=21)
    assert M.table.on_lines == 1
    M.step_and_check(4, rounding=rounding, seed=5)


@pytest.mark.parametrize("grad", ["f16", "f32"])
def test_step_of_many_ranks(grad):
    M = Model([2500, 3], 300, grad, "bf16", 32, seed=3)
    M.step_and_check(2)


@pytest.mark.parametrize("shift", [0, 1, 2, 5, 8])
def test_stochastic_rounding_bits(shift):
    M = Model(ODD, 2, "bf16", "bf16", 8, shift, seed=31)
    for step, seed in ((1, 0), (2, 2**64 - 1), ((1 << 33) + 1, 12345678901234567)):
        M.draw()
        M.step_and_check(step, rounding="stochastic", seed=seed)


def test_no_decay_no_clip_is_the_adam_step():
    """Bit for bit with zs_fused_shard_step_multi where decay and clipping are off."""
    lens = [5000, 1, 70_001]
    M = Model(lens, 4, "bf16", "bf16", 32, seed=5)
    M.decay, M.lr_scale = [0.0] * 3, [1.0] * 3
    M.table = M.upload()
    other = [Buffers(lens, torch.float32, 0).fill([x[i].clone() for i in range(3)])
             for x in (M.w, M.m, M.v)]
    par = Buffers(lens, torch.bfloat16, 0)
    chunk = 2048
    pieces = [(i, 0, sum(lens[:i]), n) for i, n in enumerate(lens)]
    nb = z.zs_mt_workspace_bytes(3, sum(-(-n // chunk) for n in lens), 4)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    ptrs = [dict(w=other[0][i], m=other[1][i], v=other[2][i], param=par[i],
                 grads=[b[i] for b in M.g]) for i in range(3)]
    t = z.zs_mt_upload(pieces, ptrs, 4, "bf16", "bf16", chunk, ws, nb)
    for step in (1, 2, 3):
        z.zs_fused_shard_step_multi(t, z.hparams(LR, B1, B2, EPS, step))
        a.zs_adamw_step_multi(M.table, a.hparams(LR, B1, B2, EPS, step))
    for i in range(3):
        for x, y in zip((M.w, M.m, M.v, M.pb), other + [par]):
            assert np.array_equal(bits_of(x[i]), bits_of(y[i]))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad_scale,sumsq,max_norm", [
    (1.0, 9.0, 1.0),              # clipped to a third
    (1.0, 0.25, 1.0),             # below the limit
    (1.0, 0.0, 1.0),
    (1.0, 4.0, 0.0),              # a norm that nothing uses
    (1 / 1024, 25.0 * 2 ** 20, 2.0),
    (-2.0, 9.0, 1.0),
])
def test_clipping(bits, grad_scale, sumsq, max_norm):
    M = Model([3000, 300], 1, "bf16", "bf16", bits, seed=6)
    M.step_and_check(3, grad_scale=grad_scale, sumsq=sumsq, max_norm=max_norm)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_nonfinite_norm(bits, bad):
    M = Model([3000, 300], 1, "bf16", "bf16", bits, seed=6)
    before = [b.flat.clone() for b in M.all()]
    sumsq = torch.tensor(bad, dtype=torch.float64, device=DEV)
    hp = a.hparams(LR, B1, B2, EPS, 3, max_norm=1.0, skip_nonfinite=True)
    a.zs_adamw_step_multi(M.table, hp, sumsq)
    for b, x in zip(M.all(), before):
        assert np.array_equal(bits_of(b.flat), bits_of(x))
    # a finite one does step
    sumsq.fill_(4.0)
    a.zs_adamw_step_multi(M.table, hp, sumsq)
    assert not np.array_equal(bits_of(M.w.flat), bits_of(before[0]))
    # without the switch an infinite norm scales the gradient to zero, NaN poisons
    M = Model([3000, 300], 1, "bf16", "bf16", bits, seed=6)
    if bad == float("inf"):
        M.step_and_check(3, sumsq=bad, max_norm=1.0, bounds=False)
    else:
        a.zs_adamw_step_multi(M.table, a.hparams(LR, B1, B2, EPS, 3, max_norm=1.0),
                              torch.tensor(bad, dtype=torch.float64, device=DEV))
        assert bool(M.w[0].isnan().all())


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_8bit_blocks_with_special_values(rounding):
    lens = [256 * 6 + 10]
    M = Model(lens, 1, "f32", "bf16", 8, seed=8)
    g = M.g[0][0]
    M.m[0].zero_(), M.v[0].zero_(), M.ms[0].zero_(), M.vs[0].zero_()
    g[:256] = 0                       # nothing seen, nothing held
    g[256:512] = 1e-35                # below what a block holds: zeros
    g[300] = -1e-36
    g[512:768] *= torch.logspace(-20, 3, 256, device=DEV)   # over the whole range of codes
    g[768] = float("inf")
    g[1024 + 7] = float("nan")
    g[1280:1536] = 1e-20              # v underflows to zero
    g[1280] = 1e-3
    g[-3:] = 0
    M.step_and_check(1, rounding=rounding, seed=3, bounds=False)
    s = M.ms[0].cpu().numpy()
    assert s[0] == 0 and s[1] == 0 and np.isnan(s[3]) and np.isnan(s[4]) and s[5] > 0
    v = ref.decode(M.v[0].cpu().numpy(), M.vs[0].cpu().numpy(), "v")
    gh = g.cpu().numpy()
    seen = (gh != 0) & (np.float32(1 - B2) * (gh * gh) > 0) & np.isfinite(v)
    seen[256:512] = False
    assert np.all(v[seen] > 0)        # a positive v stays one


def test_stochastic_rounding_keeps_the_mean_over_steps():
    """Unbiased over seeds: 5 standard deviations of a rounding that is off by
    one spacing at most."""
    n, seeds = 4096, 64
    M = Model([n], 1, "bf16", None, 8, seed=9)
    keep = [b.flat.clone() for b in M.all()]
    d = M.host(0)
    h = dict(lr=LR, decay=0.1, beta1=B1, beta2=B2, eps=EPS, step=5, gs=1.0)
    _, m, v, _ = ref.step32(ref.mean32(d["g"]), d["w"], d["m"], d["v"], h, 8)
    sums = {"m": 0.0, "v": 0.0}
    for seed in range(seeds):
        for b, x in zip(M.all(), keep):
            b.flat.copy_(x)
        a.zs_adamw_step_multi(M.table, a.hparams(LR, B1, B2, EPS, 5, rounding="stochastic", seed=seed))
        for k in sums:
            sums[k] = sums[k] + M.host(0)[k].astype(np.float64)
    for k, x in (("m", m), ("v", v)):
        top = np.repeat(np.abs(x).reshape(-1, 256).max(1), 256)
        spacing = np.maximum(np.abs(x) * 2.0 ** -ref.BITS[k],
                             top / ref.TOP[k] * 2.0 ** (ref.LEAST[k] - ref.BITS[k]))
        off = (sums[k] / seeds - x) / spacing
        # the mean over all values of a difference whose deviation is at most 1/2 each
        assert abs(off.mean()) <= 5 * 0.5 / np.sqrt(n * seeds), k
        assert np.abs(off).max() <= 6 * 0.5 / np.sqrt(seeds), k


# ---- the norm ---------------------------------------------------------------------
@pytest.mark.parametrize("grad,p,shift,store", [
    ("bf16", 1, 0, False), ("f16", 1, 1, True), ("f32", 1, 0, False), ("f32", 3, 1, True),
    ("bf16", 8, 0, True), ("f16", 5, 3, False), ("bf16", 300, 0, True)])
def test_sumsq(grad, p, shift, store):
    lens = ODD + ([3_000_001, 1_200_003] if p < 9 else [])
    M = Model(lens, p, grad, None, 32, shift, seed=40 + p, mean=store, gscale=1e-2)
    out = torch.full((3,), 7.0, dtype=torch.float64, device=DEV)
    a.zs_grad_sumsq_multi(M.table, out[1:], store_mean=store)
    means = [ref.mean32([b[i].float().cpu().numpy() for b in M.g]) for i in range(len(lens))]
    want = sum(float(np.dot(x.astype(np.float64), x.astype(np.float64))) for x in means)
    got = out.cpu().numpy()
    assert got[0] == 7.0 and got[2] == 7.0
    # both sums in double over positive terms: at most n roundings of half a step each, in fact far fewer
    assert abs(got[1] - want) <= sum(lens) * 2.0 ** -53 * want
    if store:
        for i, x in enumerate(means):
            same(M.mean[i], x, f"mean of tensor {i}")
        M.mean.check("mean")
    for b in M.g + M.all():
        b.check("buffer")
    # the same bits again; and added to what is there
    again = torch.zeros((), dtype=torch.float64, device=DEV)
    a.zs_grad_sumsq_multi(M.table, again)
    assert again.item() == got[1]
    a.zs_grad_sumsq_multi(M.table, again, accumulate=True)
    assert again.item() == got[1] + got[1]


@pytest.mark.parametrize("value,want", [(float("inf"), float("inf")), (float("nan"), float("nan")),
                                        (3e38, 9e76 * 5)])
def test_sumsq_of_large_and_nonfinite(value, want):
    M = Model([1000], 1, "f32", None, 32, seed=1)
    M.g[0][0].zero_()
    M.g[0][0][::200] = value
    out = torch.zeros((), dtype=torch.float64, device=DEV)
    a.zs_grad_sumsq_multi(M.table, out)
    assert out.isnan().item() if np.isnan(want) else out.item() == pytest.approx(want, rel=2.0 ** -23)


def test_sumsq_of_no_tensors():
    ws = torch.empty(a.zs_adamw_workspace_bytes([], 1), dtype=torch.uint8, device=DEV)
    t = a.zs_adamw_upload([], 1, "bf16", "bf16", 32, ws, ws.numel())
    out = torch.full((), 5.0, dtype=torch.float64, device=DEV)
    a.zs_grad_sumsq_multi(t, out, accumulate=True)
    assert out.item() == 5.0
    a.zs_grad_sumsq_multi(t, out)
    assert out.item() == 0.0
    a.zs_adamw_step_multi(t, a.hparams(LR, B1, B2, EPS, 1))


# ---- conversions ------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["m", "v"])
def test_every_code_decodes_and_encodes(kind):
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    dtype = torch.float8_e4m3fn if kind == "m" else torch.float8_e5m2
    for s in (1.0, 3.7e-9, 2.0 ** -100):
        scale = torch.full((1,), s, device=DEV)
        x = torch.empty(256, device=DEV)
        a.zs_state8_decode(codes, scale, 256, kind, x)
        same(x, ref.decode(codes.cpu().numpy(), np.full(1, s, np.float32), kind), f"scale {s}")
    # values on the grid and the midpoints between them, the largest present: ties to even
    grid = ref.grid_values(kind)[:128]
    grid = grid[np.isfinite(grid)]
    mid = (grid[1:] + grid[:-1]) / 2
    for vals in (grid, mid, np.nextafter(mid, np.inf), np.nextafter(mid, 0)):
        x = np.zeros(256, np.float32)
        x[:vals.size] = vals
        x[255] = ref.TOP[kind]
        if kind == "m":
            x[1:vals.size:2] *= -1
        got = torch.empty(256, dtype=torch.uint8, device=DEV)
        sc = torch.empty(1, device=DEV)
        a.zs_state8_encode(torch.from_numpy(x).to(DEV), 256, kind, got, sc)
        c, s = ref.encode(x, kind)
        same(got, c, "codes")
        same(sc, s, "scale")
        if kind == "m" or vals is grid:
            t = torch.from_numpy(x).to(dtype).view(torch.uint8).numpy()
            assert np.array_equal(t, c)


@pytest.mark.parametrize("kind", ["m", "v"])
@pytest.mark.parametrize("n", [1, 3, 255, 256, 257, 4097, 1_000_003, 2_100_000])
@pytest.mark.parametrize("shift", [0, 1])
def test_convert(kind, n, shift):
    r = np.random.default_rng(n)
    x = (r.standard_normal(n) * 10.0 ** r.uniform(-6, 1, n)).astype(np.float32)
    x = np.abs(x) if kind == "v" else x
    src = Buffers([n], torch.float32, shift).fill([x])
    codes = Buffers([n], torch.uint8, shift)
    sc = Buffers([-(-n // 256)], torch.float32, 0)
    back = Buffers([n], torch.float32, shift)
    a.zs_state8_encode(src[0], n, kind, codes[0], sc[0])
    a.zs_state8_decode(codes[0], sc[0], n, kind, back[0])
    c, s = ref.encode(x, kind)
    same(codes[0], c, "codes")
    same(sc[0], s, "scales")
    same(back[0], ref.decode(c, s, kind), "values")
    for b in (src, codes, sc, back):
        b.check("buffer")


# ---- together, on streams and in graphs ---------------------------------------------
@pytest.mark.parametrize("bits,rounding", [(32, "nearest"), (8, "stochastic")])
def test_training_steps_with_clipping(bits, rounding):
    """Norm over two tables (the mean of 4 ranks kept), then the steps from the
    stored mean, three times over."""
    lens = [3000, 500, 70_003]
    M = Model(lens, 1, "f32", "bf16", bits, seed=50, states=False)
    R = [Model(lens[i:j], 4, "bf16", None, 32, seed=51 + i, mean=True) for i, j in ((0, 2), (2, 3))]
    for i in range(3):
        M.g[0].offs  # the step's gradients are the norm's means
    src = [R[0].mean[0], R[0].mean[1], R[1].mean[0]]
    ps = M.pieces()
    for q, x in zip(ps, src):
        q["grads"] = [x]
    M.table = a.zs_adamw_upload(ps, 1, "f32", "bf16", bits, M.ws, M.ws.numel())
    sumsq = torch.zeros((), dtype=torch.float64, device=DEV)
    for step in (1, 2, 3):
        for k, r in enumerate(R):
            r.draw()
            a.zs_grad_sumsq_multi(r.table, sumsq, store_mean=True, accumulate=k > 0)
        for i, x in enumerate(src):
            M.g[0][i].copy_(x)
        M.step_and_check(step, sumsq=sumsq.item(), max_norm=0.1, rounding=rounding, seed=4)
        assert sumsq.item() > 0.01  # it did clip


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_and_replayed(bits):
    """A captured norm and step, replayed with eager work between, against the
    eager calls: every replay."""
    M, E = (Model([5000, 300, 30_001], 2, "bf16", "bf16", bits, seed=60, mean=True) for _ in range(2))
    sums = [torch.zeros((), dtype=torch.float64, device=DEV) for _ in range(2)]
    hp = a.hparams(LR, B1, B2, EPS, 9, max_norm=0.05, rounding="stochastic" if bits == 8 else "nearest",
                   seed=77)

    def both(x, out):
        a.zs_grad_sumsq_multi(x.table, out, store_mean=True)
        a.zs_adamw_step_multi(x.table, hp, out)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph):
            both(M, sums[0])
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        E.draw()
        for x, y in zip(M.g, E.g):
            x.flat.copy_(y.flat)
        graph.replay()
        both(E, sums[1])
        torch.cuda.synchronize()
        assert sums[0].item() == sums[1].item()
        for x, y in zip(M.all() + [M.mean], E.all() + [E.mean]):
            assert np.array_equal(bits_of(x.flat), bits_of(y.flat))


def test_two_streams_at_once():
    M = [Model([200_003, 5000], 1, "bf16", "bf16", 8, seed=70 + i) for i in range(2)]
    E = [Model([200_003, 5000], 1, "bf16", "bf16", 8, seed=70 + i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in M]
    sums = torch.zeros(2, dtype=torch.float64, device=DEV)
    for step in range(1, 6):
        hp = a.hparams(LR, B1, B2, EPS, step, max_norm=1.0)
        for i, (m, s) in enumerate(zip(M, streams)):
            s.wait_stream(torch.cuda.current_stream())
            a.zs_grad_sumsq_multi(m.table, sums[i], stream=s)
            a.zs_adamw_step_multi(m.table, hp, sums[i], stream=s)
    torch.cuda.synchronize()
    one = torch.zeros((), dtype=torch.float64, device=DEV)
    for m, e in zip(M, E):
        for step in range(1, 6):
            a.zs_grad_sumsq_multi(e.table, one)
            a.zs_adamw_step_multi(e.table, a.hparams(LR, B1, B2, EPS, step, max_norm=1.0), one)
        for x, y in zip(m.all(), e.all()):
            assert np.array_equal(bits_of(x.flat), bits_of(y.flat))


@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_beyond_32_bits(bits):
    """One tensor of over 2^30 (32-bit moments) or 2^31 elements: blocks at its
    start, in its middle and at its end."""
    n = 1_100_000_123 if bits == 32 else 2_300_000_123
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    g = torch.randn(n, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(1e-3)
    w = torch.randn(n, generator=gen, device=DEV).mul_(0.02)
    sd = torch.uint8 if bits == 8 else torch.float32
    m, v = torch.zeros(n, dtype=sd, device=DEV), torch.zeros(n, dtype=sd, device=DEV)
    nb = -(-n // 256)
    ms, vs = torch.zeros(nb, device=DEV), torch.zeros(nb, device=DEV)
    par = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(a.zs_adamw_workspace_bytes([n], 1), dtype=torch.uint8, device=DEV)
    index = (1 << 40) + 5
    t = a.zs_adamw_upload([dict(len=n, grads=[g], w=w, m=m, v=v, m_scale=ms, v_scale=vs, param=par,
                                weight_decay=0.1, index=index)], 1, "bf16", "bf16", bits, ws, ws.numel())
    parts = [(0, 4096), (n // 2 // 256 * 256, 4096), (n // 256 * 256 - 2048, 2048 + n % 256)]
    w0 = [w[o:o + k].cpu().numpy().copy() for o, k in parts]
    a.zs_adamw_step_multi(t, a.hparams(LR, B1, B2, EPS, 1, rounding="stochastic", seed=1))
    h = dict(lr=LR, decay=0.1, beta1=B1, beta2=B2, eps=EPS, step=1, gs=1.0)
    for (o, k), x in zip(parts, w0):
        zero = np.zeros(k, np.float32)
        ww, mm, vv, *off = ref.step32(g[o:o + k].float().cpu().numpy(), x, zero, zero, h, bits)
        if bits == 32:
            same(w[o:o + k], ww, f"w at {o}")
            same(m[o:o + k], mm, f"m at {o}")
            same(v[o:o + k], vv, f"v at {o}")
        else:
            assert np.all(np.abs(w[o:o + k].cpu().numpy() - ww.astype(np.float64)) <= off[0])
            lo, hi = ref.halves_for(k, index + o, 1, 1)
            for name, val, r, got, sc in (("m", mm, lo, m, ms), ("v", vv, hi, v, vs)):
                c, s = ref.encode(val, name, r)
                same(got[o:o + k], c, f"{name} codes at {o}")
                same(sc[o // 256:o // 256 + s.size], s, f"{name} scales at {o}")
    out = torch.zeros((), dtype=torch.float64, device=DEV)
    a.zs_grad_sumsq_multi(t, out)
    want = g.view(-1)[: n // 1024 * 1024].view(1024, -1).float().square().sum(1, dtype=torch.float64).sum()
    want = want + g[n // 1024 * 1024:].double().square().sum()
    # squares of bf16 are exact in fp32, the sums are in double
    assert abs(out.item() - want.item()) <= 1e-10 * want.item()


@pytest.mark.parametrize("bits,rounding", [(32, "nearest"), (8, "stochastic")])
def test_captured_steps_follow_a_step_table(bits, rounding):
    """A graph of norm, step and advance, replayed with eager work between:
    each replay the next step of a learning-rate schedule; a step whose norm is
    not finite changes and counts nothing; past the end nothing moves."""
    lens = [5000, 300, 30_001]
    M, E = (Model(lens, 2, "bf16", "bf16", bits, seed=80) for _ in range(2))
    lrs = [1e-3 / k for k in (1, 2, 3, 4, 5)]
    kw = dict(max_norm=0.05, rounding=rounding, seed=9, skip_nonfinite=True)
    hp = a.hparams(1.0, B1, B2, EPS, 41, **kw)
    buf = torch.empty(a.zs_adamw_steps_bytes(len(lrs)), dtype=torch.uint8, device=DEV)
    steps = a.zs_adamw_steps_init(hp, len(lrs), buf, buf.numel(), lrs=lrs)
    sums = [torch.zeros((), dtype=torch.float64, device=DEV) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph):
            a.zs_grad_sumsq_multi(M.table, sums[0])
            a.zs_adamw_step_multi_dev(M.table, steps, hp, sums[0])
            a.zs_adamw_steps_advance(steps, sums[0])
    torch.cuda.current_stream().wait_stream(side)
    done = 0
    for i in range(8):
        E.draw()
        if i == 2:
            E.g[1][2][7] = float("inf")
        for x, y in zip(M.g, E.g):
            x.flat.copy_(y.flat)
        graph.replay()
        a.zs_grad_sumsq_multi(E.table, sums[1])
        if i != 2 and done < len(lrs):
            a.zs_adamw_step_multi(E.table, a.hparams(lrs[done], B1, B2, EPS, 41 + done, **kw), sums[1])
            done += 1
        cursor, exhausted = a.zs_adamw_steps_status(steps)
        # an advance past the end still moves the cursor, as zs_step_table_advance's does
        assert cursor == (i + 1 if i < 2 else i) and exhausted == (1 if i >= 6 else 0)
        for x, y in zip(M.all(), E.all()):
            assert np.array_equal(bits_of(x.flat), bits_of(y.flat)), f"replay {i}"
    assert done == len(lrs)


# ---- calls that nothing above makes ---------------------------------------------------
def test_most_ranks_and_shared_gradients():
    """ZS_MAX_P ranks; then ranks and tensors that all read one buffer."""
    M = Model([700, 1], z.ZS_MAX_P, "bf16", "bf16", 8, seed=90)
    M.step_and_check(2, bounds=False)
    M = Model([3000, 3000], 3, "f32", "f16", 32, seed=91)
    ps = M.pieces()
    one = M.g[0][0]
    for q in ps:
        q["grads"] = [one] * 3
    M.table = a.zs_adamw_upload(ps, 3, "f32", "f16", 32, M.ws, M.ws.numel())
    for b in M.g:
        for i in range(2):
            b[i].copy_(one)
    M.step_and_check(2)
    out = torch.zeros((), dtype=torch.float64, device=DEV)
    a.zs_grad_sumsq_multi(M.table, out)
    x = ref.mean32([one.cpu().numpy()] * 3).astype(np.float64)
    assert abs(out.item() - 2 * np.dot(x, x)) <= 6000 * 2.0 ** -53 * out.item()


def test_nonfinite_gradients_stay_in_their_elements():
    """32-bit moments: IEEE rules element by element."""
    M = Model([1000], 1, "f32", "bf16", 32, seed=92)
    g = M.g[0][0]
    g[5], g[6], g[7], g[999] = float("inf"), float("-inf"), float("nan"), 3e38
    M.step_and_check(2, bounds=False)
    bad = ~np.isfinite(M.w[0].cpu().numpy())
    assert bad[[5, 6, 7]].all() and bad.sum() == 3


def test_values_outside_the_copy_and_zero_moments():
    M = Model([600], 1, "bf16", "f16", 32, seed=93, states=False)
    M.w[0][:3] = torch.tensor([1e6, -1e6, 1e-9], device=DEV)
    M.g[0][0].zero_()
    M.step_and_check(1, bounds=False)  # 0 / (0 + eps) moves nothing; the copy overflows and underflows
    assert M.pb[0][:2].isinf().all() and M.pb[0][2] == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero_states(bits):
    """Codes and scales all zero are the zero state; step 1 moves by lr where the
    gradient is far above eps."""
    M = Model([5000, 10], 1, "bf16", "bf16", bits, seed=94, states=False, gscale=1.0)
    M.decay = [0.0, 0.0]
    M.table = M.upload()
    w0, g = M.w[0].clone(), M.g[0][0].float()
    M.step_and_check(1)
    moved = (M.w[0] - w0)[g.abs() > 1e-2]
    # lr * (1 +- 8 half steps), and w's own rounding (w < 1/8: half a step is 2^-28)
    assert float((moved.abs() - LR).abs().max()) <= LR * 8 * ref.U + 2.0 ** -27


def test_current_stream_is_taken():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert z._stream(None) == s.cuda_stream
    assert z._stream(None) == torch.cuda.current_stream().cuda_stream
    assert z._stream(s) == s.cuda_stream and z._stream(5) == 5


def test_two_graphs_replayed_on_two_streams():
    """Two captured loops with tables of their own, replayed at once."""
    sets = []
    for i in range(2):
        M, E = (Model([100_003, 700], 1, "bf16", "bf16", 8, seed=95 + i) for _ in range(2))
        out = torch.zeros((), dtype=torch.float64, device=DEV)
        hp = a.hparams(LR, B1, B2, EPS, 3, max_norm=1.0, rounding="stochastic", seed=i)
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph):
                a.zs_grad_sumsq_multi(M.table, out)
                a.zs_adamw_step_multi(M.table, hp, out)
        sets.append((M, E, out, hp, graph, s))
    torch.cuda.synchronize()
    for _ in range(3):
        for M, E, out, hp, graph, s in sets:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for M, E, out, hp, graph, s in sets:
        one = torch.zeros_like(out)
        for _ in range(3):
            a.zs_grad_sumsq_multi(E.table, one)
            a.zs_adamw_step_multi(E.table, hp, one)
        assert one.item() == out.item()
        for x, y in zip(M.all(), E.all()):
            assert np.array_equal(bits_of(x.flat), bits_of(y.flat))


def test_moments_move_between_the_forms():
    """32-bit moments encoded, stepped in 8 bits, decoded and stepped in 32."""
    n = 5000
    A, B = Model([n], 1, "bf16", "bf16", 32, seed=97), Model([n], 1, "bf16", "bf16", 8, seed=97)
    a.zs_state8_encode(A.m[0], n, "m", B.m[0], B.ms[0])
    a.zs_state8_encode(A.v[0], n, "v", B.v[0], B.vs[0])
    B.w[0].copy_(A.w[0])
    B.step_and_check(7, rounding="stochastic", seed=1)
    a.zs_state8_decode(B.m[0], B.ms[0], n, "m", A.m[0])
    a.zs_state8_decode(B.v[0], B.vs[0], n, "v", A.v[0])
    A.w[0].copy_(B.w[0])
    A.step_and_check(8)
    for b in A.all() + B.all():
        b.check("buffer")


def test_default_rounding_follows_a_run():
    """200 steps of 8-bit moments with the binding's own choice of rounding: the
    mean of v stays at the square that it averages."""
    n, steps, beta2 = 8192, 200, 0.95
    M = Model([n], 1, "f32", None, 8, seed=98, states=False)
    g = M.g[0][0]
    g.fill_(2.5e-6 ** 0.5)
    g[::256] = 0.1  # holds each block's scale
    seen = np.arange(n) % 256 != 0
    want = float(g[1]) ** 2 * (1 - beta2 ** steps)
    for t in range(1, steps + 1):
        a.zs_adamw_step_multi(M.table, a.hparams(LR, B1, beta2, EPS, t, seed=6))
    v = M.host(0)["v"][seen].astype(np.float64)
    # five deviations of the mean, and 2^-17 of a spacing (v / 4 at most) at each step; rounded to nearest, all of
    # them end on one code, 2.3% off, with no deviation
    assert abs(v.mean() - want) <= 5 * v.std() / np.sqrt(v.size) + want * (2.0 ** -19 / (1 - beta2) + 1e-4)


@pytest.mark.parametrize("p", [1, 3])
def test_pieces_of_a_tensor_get_the_whole_ones_bits(p):
    """A tensor stepped whole, and cut at multiples of 256 into pieces whose
    indexes match: the same weights, codes and scales.  Cut elsewhere, a piece's
    random bits are those of its own fours."""
    n, cuts = 9000, [0, 256, 1280, 8192, 9000]
    M, E = (Model([n], p, "bf16", "bf16", 8, seed=99) for _ in range(2))
    q = E.pieces()[0]
    parts = []
    for lo, hi in zip(cuts, cuts[1:]):
        b = slice(lo // 256, -(-hi // 256))
        parts.append(dict(q, len=hi - lo, grads=[x[lo:hi] for x in q["grads"]], index=q["index"] + lo,
                          **{k: q[k][lo:hi] for k in ("w", "m", "v", "param")},
                          **{k: q[k][b] for k in ("m_scale", "v_scale")}))
    ws = torch.empty(a.zs_adamw_workspace_bytes([x["len"] for x in parts], p), dtype=torch.uint8, device=DEV)
    table = a.zs_adamw_upload(parts, p, "bf16", "bf16", 8, ws, ws.numel())
    hp = a.hparams(LR, B1, B2, EPS, 12, rounding="stochastic", seed=21)
    a.zs_adamw_step_multi(M.table, hp)
    a.zs_adamw_step_multi(table, hp)
    for x, y in zip(M.all(), E.all()):
        assert np.array_equal(bits_of(x.flat), bits_of(y.flat))
    N = Model([6, n - 6], p, "bf16", "bf16", 8, seed=99)
    N.index = [M.index[0], M.index[0] + 6]
    N.table = N.upload()
    N.step_and_check(12, rounding="stochastic", seed=21)


def norm_and_means(M, launches):
    """`launches` sums of squares in a row (the mean kept if M has it) against the
    exact sum of the fp32 means' squares, which are exact in double.  The sizes
    here put fewer than 64 roundings between an element and the sum: 32 on its
    lane, 6 + 8 in its workgroup, as many in the join, one for what is there."""
    means = [ref.mean32([b[i].float().cpu().numpy() for b in M.g]) for i in range(len(M.lens))]
    want = math.fsum(float(s) for x in means for s in x.astype(np.float64) ** 2)
    out = torch.full((launches + 2,), 7.0, dtype=torch.float64, device=DEV)
    for k in range(launches):
        if M.mean:
            M.mean.fill([torch.full((n,), -1.0) for n in M.lens])
        a.zs_grad_sumsq_multi(M.table, out[k + 1:], store_mean=bool(M.mean))
        if M.mean:
            for i, x in enumerate(means):
                same(M.mean[i], x, f"mean of tensor {i}")
            M.mean.check("mean")
    got = out.cpu().numpy()
    assert got[0] == 7.0 and got[-1] == 7.0
    assert abs(got[1] - want) <= 64 * 2.0 ** -53 * want
    assert np.all(got[1:-1] == got[1])
    a.zs_grad_sumsq_multi(M.table, out, accumulate=True)
    assert out[0].item() == 7.0 + got[1]
    for b in M.g + M.all():
        b.check("buffer")


@pytest.mark.parametrize("grad,store,shift", [
    ("bf16", False, 0), ("bf16", True, 3), ("f16", True, 0), ("f16", False, 1), ("f32", True, 1), ("f32", False, 0)])
@pytest.mark.parametrize("lens", [[9 * 1024], [5, 1, 2050], [100_003, 5, 700, 257], [300_001, 300_002]])
def test_sumsq_of_one_rank_in_one_launch(grad, store, shift, lens):
    """2 to 64 workgroups that add their sums in the launch."""
    norm_and_means(Model(lens, 1, grad, None, 32, shift, seed=100, mean=store, gscale=1e-2), 4)


@pytest.mark.parametrize("grad,store", [("bf16", True), ("f32", False)])
@pytest.mark.parametrize("entries", [1023, 1024, 1025])
def test_sumsq_where_one_launch_becomes_two(grad, store, entries):
    n = 1023 * 1024 + {1023: 0, 1024: 1, 1025: 1025}[entries]
    M = Model([n], 1, grad, None, 32, None, seed=101, mean=store, gscale=1e-2)
    assert M.table.nchunks == entries
    norm_and_means(M, 2)


@pytest.mark.parametrize("p,grad,store,shift,lens", [
    (2, "bf16", True, 1, [61 * 1024, 1000]), (9, "f16", False, 0, [61 * 1024, 1000]),  # one
    (2, "bf16", False, 0, [66 * 1024]), (9, "f16", True, 3, [66 * 1024]),              # two
    (17, "f16", True, 3, [300_001, 7]), (17, "f16", False, 0, [300_001, 7]),
    (64, "bf16", True, 0, [200_000, 100_003]), (64, "bf16", False, 5, [200_000, 100_003])])
def test_sumsq_of_ranks_in_one_launch_and_two(p, grad, store, shift, lens):
    M = Model(lens, p, grad, None, 32, shift, seed=102, mean=store, gscale=1e-2)
    assert (M.table.nchunks <= 64) == (sum(lens) < 64 * 1024)
    norm_and_means(M, 2)
