"""Host-side tests of the AdamW operators' C ABI (no GPU, no kernel launched):
symbols, sizes, and the refusal of every bad argument before anything reaches
the device; and the numpy reference that the GPU tests use, against torch."""

import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import adamw_ref as ref
from adam_zs_shard_amd import zsadamw as a
from adam_zs_shard_amd import zshard as z

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "zsadamw.h")
FAKE = 1 << 40
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: CPU-only test")


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(zs_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(a.EXPORTS)
    for n in names:
        assert hasattr(a.lib(), n), n


def test_workspace_bytes():
    need = a.zs_adamw_workspace_bytes
    assert need([], 1) > 0
    assert need([1], 1) >= 128 + 8
    assert need([5000, 7], 8) - need([5000, 7], 1) >= 0
    assert need([2048 * 100], 1) >= 100 * 128
    assert need([10**9], 1) < 10**9 // 8192 * 128 + 4096 * 16
    # short tensors: entries of their own size
    assert need([1000] * 10_000, 1) < 10_000 * (2 * 128 + 8) + 4096 * 16
    for bad in ([0], [-1], [1 << 61], [1 << 59, 1 << 59, 1 << 59]):
        assert need(bad, 1) == 0
    assert need([5], 0) == 0 and need([5], z.ZS_MAX_P + 1) == 0
    assert a.lib().zs_adamw_workspace_bytes(None, 1, 1) == 0
    # more workgroups than one launch counts
    assert need([1 << 40], 1) == 0


def _piece(i=0, n=1000, p=2, **over):
    base = FAKE + (i << 34)
    q = dict(len=n, w=base, m=base + (1 << 30), v=base + (2 << 30), m_scale=base + (3 << 30),
             v_scale=base + (4 << 30), param=base + (5 << 30), g_mean=base + (6 << 30),
             grads=[base + (8 << 30) + (r << 28) for r in range(p)], weight_decay=0.1)
    q.update(over)
    return q


WS = FAKE + (1 << 44)


def _upload(pieces, p=2, gdt="bf16", pdt="bf16", bits=32, ws=WS, nbytes=1 << 20):
    try:
        a.zs_adamw_upload(pieces, p, gdt, pdt, bits, ws, nbytes, stream=0)
    except z.ZsError as e:
        return e.status
    return z.ZS_OK


@no_device
@pytest.mark.parametrize("over,status", [
    (dict(len=0), z.ZS_ERR_ARG), (dict(len=-5), z.ZS_ERR_ARG), (dict(len=1 << 61), z.ZS_ERR_ARG),
    (dict(index=-1), z.ZS_ERR_ARG), (dict(weight_decay=-0.1), z.ZS_ERR_ARG),
    (dict(weight_decay=float("nan")), z.ZS_ERR_ARG), (dict(lr_scale=float("inf")), z.ZS_ERR_ARG),
    (dict(w=None), z.ZS_ERR_NULL), (dict(m=None), z.ZS_ERR_NULL), (dict(v=None), z.ZS_ERR_NULL),
    (dict(param=None), z.ZS_ERR_NULL), (dict(grads=[FAKE, None]), z.ZS_ERR_NULL),
    (dict(w=FAKE + 2), z.ZS_ERR_ARG), (dict(param=FAKE + (5 << 30) + 1), z.ZS_ERR_ARG),
    (dict(grads=[FAKE + 1, FAKE + (1 << 28)]), z.ZS_ERR_ARG),
    (dict(m=FAKE + 3996), z.ZS_ERR_ALIAS),          # the last element of w
    (dict(param=FAKE + (1 << 30) + 3998), z.ZS_ERR_ALIAS),
    (dict(g_mean=FAKE + (2 << 30)), z.ZS_ERR_ALIAS),
    (dict(grads=[FAKE + 2000, FAKE + (9 << 30)]), z.ZS_ERR_ALIAS),
    (dict(w=WS + 64), z.ZS_ERR_ALIAS),
])
def test_upload_refuses_pieces(over, status):
    assert _upload([_piece(**over)]) == status
    assert _upload([_piece(1), _piece(**over)]) == status


@no_device
def test_upload_refuses_arguments():
    q = [_piece()]
    assert _upload(q, bits=16) == z.ZS_ERR_ARG
    assert _upload(q, gdt=4) == z.ZS_ERR_DTYPE and _upload(q, pdt=3) == z.ZS_ERR_DTYPE
    assert _upload(q, ws=None) == z.ZS_ERR_NULL
    assert _upload(q, ws=WS + 128) == z.ZS_ERR_CAPACITY
    assert _upload(q, nbytes=a.zs_adamw_workspace_bytes([1000], 2) - 1) == z.ZS_ERR_CAPACITY
    assert _upload([_piece(m_scale=None)], bits=8) == z.ZS_ERR_NULL
    assert _upload([_piece(v_scale=None)], bits=8) == z.ZS_ERR_NULL
    # the fourth scale of m meets v's codes
    assert _upload([_piece(m_scale=FAKE + (2 << 30) - 12)], bits=8) == z.ZS_ERR_ALIAS
    assert _upload([_piece(p=0)], p=0) == z.ZS_ERR_ARG
    many = [_piece(p=z.ZS_MAX_P + 1)]
    assert _upload(many, p=z.ZS_MAX_P + 1) == z.ZS_ERR_ARG
    # two tensors that share one gradient may; two that share a weight may not
    assert _upload([_piece(), _piece(1, w=FAKE)]) == z.ZS_ERR_ALIAS
    assert _upload([_piece(len=1 << 40)], bits=0) == z.ZS_ERR_RANGE
    with pytest.raises(ValueError):
        a.zs_adamw_upload([_piece(p=3)], 2, "bf16", "bf16", 32, WS, 1 << 20, stream=0)
    assert a.lib().zs_adamw_upload(None, 1, 1, 1, 1, 32, WS, 1 << 20, None,
                                   C.byref(a.zs_adamw_table())) == z.ZS_ERR_NULL


def _table(**over):
    t = a.zs_adamw_table(WS, 4, 8192, 2, 2, z.ZS_BF16, z.ZS_BF16, 32, 1, 0, 0)
    for k, x in over.items():
        setattr(t, k, x)
    return t


HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1)


@no_device
@pytest.mark.parametrize("over", [
    dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")),
    dict(eps=float("inf")), dict(eps=-1e-8), dict(step=0), dict(grad_scale=0.0),
    dict(grad_scale=float("inf")), dict(max_norm=-1.0), dict(max_norm=float("inf")),
    dict(rounding=2), dict(skip_nonfinite=2)])
def test_step_refuses_hparams(over):
    hp = a.hparams(**{**HP, **over})
    assert a.zs_adamw_step_multi(_table(), hp, FAKE, stream=0, check=False) == z.ZS_ERR_ARG


@no_device
def test_step_and_sumsq_refuse_tables():
    hp = a.hparams(**HP)

    def step(t, h=hp, sumsq=None):
        return a.zs_adamw_step_multi(t, h, sumsq, stream=0, check=False)

    def norm(t, sumsq=FAKE, **k):
        return a.zs_grad_sumsq_multi(t, sumsq, stream=0, check=False, **k)

    for over, st in ((dict(workspace=None), z.ZS_ERR_NULL), (dict(p=0), z.ZS_ERR_ARG),
                     (dict(p=z.ZS_MAX_P + 1), z.ZS_ERR_ARG), (dict(npieces=-1), z.ZS_ERR_ARG),
                     (dict(nchunks=1), z.ZS_ERR_ARG), (dict(nchunks=1 << 24), z.ZS_ERR_ARG),
                     (dict(chunk_elems=100), z.ZS_ERR_ARG), (dict(state_bits=16), z.ZS_ERR_ARG),
                     (dict(grad_dtype=4), z.ZS_ERR_DTYPE), (dict(param_dtype=3), z.ZS_ERR_DTYPE)):
        assert step(_table(**over)) == st and norm(_table(**over)) == st, over
    assert step(_table(state_bits=0)) == z.ZS_ERR_ARG
    assert step(_table(), a.hparams(**HP, max_norm=1.0)) == z.ZS_ERR_NULL
    assert step(_table(), a.hparams(**HP, skip_nonfinite=True)) == z.ZS_ERR_NULL
    assert step(_table(), a.hparams(**HP, max_norm=1.0), FAKE + 4) == z.ZS_ERR_ARG
    assert a.lib().zs_adamw_step_multi(None, C.byref(hp), None, None) == z.ZS_ERR_NULL
    assert a.lib().zs_adamw_step_multi(C.byref(_table()), None, None, None) == z.ZS_ERR_NULL
    assert norm(_table(), None) == z.ZS_ERR_NULL and norm(_table(), FAKE + 4) == z.ZS_ERR_ARG
    assert norm(_table(has_mean=0), store_mean=True) == z.ZS_ERR_NULL
    assert norm(_table(), store_mean=2) == z.ZS_ERR_ARG
    assert norm(_table(), accumulate=2) == z.ZS_ERR_ARG
    # a step over no tensors is no launch
    assert step(_table(nchunks=0, npieces=0)) == z.ZS_OK


@no_device
def test_convert_refuses():
    x, c, s = FAKE, FAKE + (1 << 30), FAKE + (2 << 30)
    for enc in (True, False):
        def call(x=x, n=1000, kind="m", c=c, s=s):
            if enc:
                return a.zs_state8_encode(x, n, kind, c, s, stream=0, check=False)
            return a.zs_state8_decode(c, s, n, kind, x, stream=0, check=False)

        assert call(n=0) == z.ZS_OK and call(n=-1) == z.ZS_ERR_ARG
        assert call(n=1 << 61) == z.ZS_ERR_RANGE and call(kind=2) == z.ZS_ERR_ARG
        assert call(x=None) == call(c=None) == call(s=None) == z.ZS_ERR_NULL
        assert call(x=x + 2) == call(s=s + 1) == z.ZS_ERR_ARG
        assert call(c=x + 3999) == call(s=c + 996) == call(s=x) == z.ZS_ERR_ALIAS


# ---- the reference itself -------------------------------------------------------
@pytest.mark.parametrize("kind,dtype", [("m", torch.float8_e4m3fn), ("v", torch.float8_e5m2)])
def test_reference_grid_is_the_types(kind, dtype):
    t = torch.arange(256, dtype=torch.uint8).view(dtype).float().numpy()
    assert np.array_equal(ref.grid_values(kind).astype(np.float32), t, equal_nan=True)
    x = np.random.default_rng(1).standard_normal(40_000).astype(np.float32) ** 3
    x = np.abs(x) if kind == "v" else x
    codes, scales = ref.encode(x, kind)
    pad = np.zeros(-(-x.size // 256) * 256, np.float32)
    pad[:x.size] = x
    most = np.abs(pad.reshape(-1, 256)).max(1, keepdims=True)
    y = torch.from_numpy(np.minimum(pad.reshape(-1, 256) * (np.float32(ref.TOP[kind]) / most),
                                    np.float32(ref.TOP[kind]))).to(dtype)
    same = y.view(torch.uint8).numpy().reshape(-1)[:x.size] == codes
    assert np.all(same | ((codes == 1) & (kind == "v")))
    # a value is off by half its grid's spacing at most, plus the two products' roundings
    bound = 2.0 ** -(ref.BITS[kind] + 1) + 4 * ref.U
    big = np.abs(pad.reshape(-1, 256)) >= most * 2.0 ** (ref.LEAST[kind] - 8 + (kind == "v") * -7)
    back = ref.decode(codes, scales, kind)
    sel = big.reshape(-1)[:x.size] & (x != 0)
    assert np.all(np.abs(back[sel] - x[sel]) <= bound * np.abs(x[sel]))


def test_reference_philox_known_answers():
    # seven rounds by hand on Python integers
    def one(c, k):
        for _ in range(7):
            x, y = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(y >> 32) ^ c[1] ^ k[0], y & 0xFFFFFFFF, (x >> 32) ^ c[3] ^ k[1], x & 0xFFFFFFFF]
            k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
        return c

    seed, step = 0x123456789ABCDEF0, (3 << 32) + 7
    idx = np.array([0, 4, (5 << 32) + 8], np.uint64)
    got = ref.philox(idx, step, seed)
    for i, row in zip(idx.tolist(), got):
        want = one([i & 0xFFFFFFFF, i >> 32, step & 0xFFFFFFFF, step >> 32],
                   [seed & 0xFFFFFFFF, seed >> 32])
        assert [int(x) for x in row] == want


def test_reference_random_rounding_keeps_the_mean():
    """All 2^16 random halves of a value: the mean stored is the value to the
    16 bits' own half step, 2^-17 of the grid's spacing."""
    halves = np.arange(1 << 16, dtype=np.uint32)
    for kind in ("m", "v"):
        for x in (1.07, 0.3, 2.0 ** -9, 3.3e-5):
            row = np.full(256, x, np.float32)
            row[0] = 1.0 if x < 1 else x  # the block's largest value
            mean = 0.0
            for k in range(0, 1 << 16, 255):
                h = np.zeros(256, np.uint32)
                part = halves[k:k + 255]
                h[1:1 + part.size] = part
                c, s = ref.encode(row, kind, h)
                mean += ref.decode(c, s, kind)[1:1 + part.size].astype(np.float64).sum()
            mean /= 1 << 16
            top = float(row[0])
            spacing = max(2.0 ** -ref.BITS[kind] * x, top / ref.TOP[kind] * 2.0 ** (ref.LEAST[kind] - ref.BITS[kind]))
            assert abs(mean - x) <= spacing * (2.0 ** -17 + 2.0 ** -16) + 8 * ref.U * x, (kind, x)


def test_reference_step_is_torch_adamw():
    rng = np.random.default_rng(3)
    n, t0 = 4000, 1
    w = rng.standard_normal(n).astype(np.float32) * 0.02
    p = torch.nn.Parameter(torch.from_numpy(w.astype(np.float64)))
    opt = torch.optim.AdamW([p], lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    m = np.zeros(n, np.float32)
    v = np.zeros(n, np.float32)
    m64, v64, w64 = (x.astype(np.float64) for x in (m, v, w))
    slack = np.zeros(n)
    for t in range(t0, t0 + 6):
        g = rng.standard_normal(n).astype(np.float32)
        p.grad = torch.from_numpy(g.astype(np.float64))
        opt.step()
        h = dict(lr=1e-3, decay=0.1, beta1=0.9, beta2=0.95, eps=1e-8, step=t, gs=1.0)
        w64, m64, v64, bw, _, _ = ref.step64([g], w64, m64, v64, h)
        w, m, v = ref.step32(g, w, m, v, h)
        slack += bw + 1e-3 * 1e-5  # what earlier steps' roundings of m and v do to this one's quotient
        # torch decays first and moves then: lr^2 * decay * u apart
        assert np.all(np.abs(p.detach().numpy() - w64) <= t * 1e-3 * 1e-3 * 0.1 * 12)
        assert np.all(np.abs(w - w64) <= slack)


@no_device
def test_step_tables_refuse():
    hp = a.hparams(**HP)
    assert a.zs_adamw_steps_bytes(0) == a.zs_adamw_steps_bytes(z.ZS_MAX_TABLE_STEPS + 1) == 0
    assert a.zs_adamw_steps_bytes(1) % 256 == 0 and a.zs_adamw_steps_bytes(1000) >= 1000 * 56

    def init(hp=hp, n=10, dev=FAKE, nb=1 << 16, **k):
        try:
            a.zs_adamw_steps_init(hp, n, dev, nb, stream=0, **k)
        except z.ZsError as e:
            return e.status
        return z.ZS_OK

    assert init(n=0) == init(n=-1) == init(n=z.ZS_MAX_TABLE_STEPS + 1) == z.ZS_ERR_ARG
    assert init(a.hparams(**{**HP, "beta2": 1.0})) == z.ZS_ERR_ARG
    assert init(a.hparams(**{**HP, "step": 2**63 - 5})) == z.ZS_ERR_RANGE
    assert init(dev=None) == z.ZS_ERR_NULL and init(dev=FAKE + 64) == z.ZS_ERR_CAPACITY
    assert init(nb=a.zs_adamw_steps_bytes(10) - 1) == z.ZS_ERR_CAPACITY
    assert init(n=2, lrs=[1e-3, float("nan")]) == z.ZS_ERR_ARG
    with pytest.raises(ValueError):
        init(n=3, lrs=[1e-3])

    def steps(**over):
        s = a.zs_adamw_steps(FAKE, 1, 10, 0)
        for k, x in over.items():
            setattr(s, k, x)
        return s

    for over, st in ((dict(dev=None), z.ZS_ERR_NULL), (dict(nsteps=0), z.ZS_ERR_ARG),
                     (dict(reserved=1), z.ZS_ERR_ARG)):
        s = steps(**over)
        assert a.zs_adamw_steps_advance(s, stream=0, check=False) == st
        assert a.zs_adamw_step_multi_dev(_table(), s, hp, stream=0, check=False) == st
        with pytest.raises(z.ZsError):
            a.zs_adamw_steps_status(s, stream=0)
    assert a.zs_adamw_steps_advance(steps(), FAKE + 4, stream=0, check=False) == z.ZS_ERR_ARG
    assert a.zs_adamw_step_multi_dev(_table(state_bits=0), steps(), hp, stream=0,
                                     check=False) == z.ZS_ERR_ARG
    assert a.zs_adamw_step_multi_dev(_table(), steps(), a.hparams(**HP, max_norm=1.0), stream=0,
                                     check=False) == z.ZS_ERR_NULL


# ---- rounding over a run ----------------------------------------------------------
def test_moments_round_at_random_unless_told():
    assert a.hparams(**HP).rounding == a.ZS_ROUND_STOCHASTIC
    assert a.hparams(**HP, rounding="nearest").rounding == a.ZS_ROUND_NEAREST


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
def test_rounding_of_v_over_a_run(beta2):
    """300 steps of v from 1e-6 in blocks whose scale another element holds: with
    a constant gradient, and with none.  Rounded to nearest, v never comes near
    the square that it averages, and never decays; at random it follows both in
    the mean."""
    n, steps, u = 2048, 300, ref.U
    g = np.full(n, np.sqrt(2.5e-6), np.float32)
    g[1::2] = 0.0
    g[::256] = 0.1
    start = np.full(n, 1e-6, np.float32)
    start[::256] = 1e-2
    seen, gone = np.arange(n) % 2 == 0, np.arange(n) % 2 == 1
    seen[::256] = False
    want = np.float64(beta2) ** steps * 1e-6 + (1 - np.float64(beta2) ** steps) * g.astype(np.float64) ** 2
    got = {}
    for rounding in a.ROUNDINGS:
        codes, scales = ref.encode(start, "v")
        first = ref.decode(codes, scales, "v")
        if rounding == "stochastic":  # its start as it is: the mean of many roundings
            codes, scales = ref.encode(start, "v", ref.halves_for(n, 0, 0, 5)[1])
        for t in range(1, steps + 1):
            v = np.float32(beta2) * ref.decode(codes, scales, "v") + np.float32(1 - beta2) * (g * g)
            halves = ref.halves_for(n, 0, t, 5)[1] if rounding == "stochastic" else None
            codes, scales = ref.encode(v, "v", halves)
        got[rounding] = ref.decode(codes, scales, "v").astype(np.float64)
    # the scale's roundings alone move a code that stays: four a step, of a half step each
    near = got["nearest"]
    assert np.all(np.abs(near[gone] - first[gone]) <= 4 * steps * u * first[gone])
    assert np.all((1 - beta2) * (want[seen] - near[seen]) <= near[seen] / 8)
    assert np.all(near[seen] < 0.6 * 2.5e-6)
    for which in (seen, gone):
        x, w = got["stochastic"][which], want[which][0]
        # five deviations of the mean; 16 bits leave 2^-17 of a spacing, v / 4 at most, at each step; v itself
        # is at least the smallest code
        least = 1e-2 * 2.0 ** -16 / 57344
        slack = 2.0 ** -19 * max(w, 1e-6) / (1 - beta2) + 4 * steps * u * max(w, 1e-6)
        assert abs(x.mean() - w) <= 5 * x.std() / np.sqrt(x.size) + slack + (least if w < 64 * least else 0)


def test_random_bits_of_cut_tensors():
    """Fours of elements share a counter and are counted from the piece's first
    one: a cut at a multiple of 4 leaves every element its bits."""
    n, index, step, seed = 64, (1 << 33) + 6, 3, 11
    whole = np.stack(ref.halves_for(n, index, step, seed))
    for cut in (4, 8, 60):
        first, rest = ref.halves_for(cut, index, step, seed), ref.halves_for(n - cut, index + cut, step, seed)
        assert np.array_equal(np.concatenate([first, rest], 1), whole)
    for cut in (1, 6, 63):
        rest = np.stack(ref.halves_for(n - cut, index + cut, step, seed))
        assert not np.any(np.all(rest == whole[:, cut:], 0))


def test_random_rounding_of_v_below_the_smallest_code():
    """A positive v below the smallest code always gets it; from there on, and
    for m everywhere, the mean is kept."""
    halves = np.arange(255, dtype=np.uint32) * 257
    least = 2.0 ** -16 / 57344
    for x, kept in ((1e-12, False), (0.9 * least, False), (1.5 * least, True)):
        row = np.full(256, x, np.float32)
        row[0] = 1.0
        c, s = ref.encode(row, "v", np.concatenate([np.zeros(1, np.uint32), halves]))
        back = ref.decode(c, s, "v")[1:].astype(np.float64)
        assert np.all(c[1:] >= 1)
        # 255 evenly spread halves: the share that rounds up is off by one of them at most
        assert (abs(back.mean() - x) <= least / 254) == kept
        assert kept or np.all(c[1:] == 1)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("decay,lr_scale", [(0.1, 1.0), (0.01, 1.0), (0.5, 0.5), (0.0, 2.0)])
def test_reference_definition_is_torch_adamw(bits, decay, lr_scale):
    """step64 against torch's AdamW in 64 bits, on weights up to some tens: both
    are w - lr*u - lr*decay*w, so only 64-bit roundings lie between them."""
    rng = np.random.default_rng(4)
    n, lr, b1, b2, u64 = 3000, 1e-3, 0.9, 0.95, 2.0 ** -53
    w = rng.standard_normal(n) * 10.0 ** rng.uniform(-2, 1.5, n)
    p = torch.nn.Parameter(torch.from_numpy(w.copy()))
    opt = torch.optim.AdamW([p], lr=lr * lr_scale, betas=(b1, b2), eps=1e-8, weight_decay=decay)
    m, v, size, bound = np.zeros(n), np.zeros(n), np.zeros(n), np.zeros(n)
    for t in range(1, 9):
        g = rng.standard_normal(n) * 1e-2
        p.grad = torch.from_numpy(g.copy())
        opt.step()
        h = dict(lr=lr * lr_scale, decay=decay, beta1=b1, beta2=b2, eps=1e-8, step=t, gs=1.0)
        w, m, v, *_ = ref.step64([g], w, m, v, h, bits)
        # on each side m is off by 4 roundings of its terms' sizes at each step (5 t in all), v by as many of itself;
        # the quotient has the corrections, a root, a sum and a division besides, the weight two products and two
        # sums: 40 (t + 1) and 8 cover both sides
        size = b1 * size + (1 - b1) * np.abs(g)
        most = size / (1 - b1 ** t) / (np.sqrt(v / (1 - b2 ** t)) + 1e-8)
        bound += u64 * (40 * (t + 1) * lr * lr_scale * most + 8 * np.abs(w))
        assert np.all(np.abs(p.detach().numpy() - w) <= bound)
    # what a decay or a learning rate that is a tenth off would move is far above
    assert np.all(bound < 1e-9 * (lr * lr_scale * most + np.abs(w)))
    state = opt.state[p]
    assert np.all(np.abs(state["exp_avg"].numpy() - m) <= 100 * u64 * size)
    assert np.all(np.abs(state["exp_avg_sq"].numpy() - v) <= 100 * u64 * v)


@pytest.mark.parametrize("bits", [32, 8])
def test_reference_sequence_stays_within_the_definition(bits):
    """step32 and its bounds against step64, several ranks, clipped and scaled."""
    rng = np.random.default_rng(5)
    n = 3000
    w = (rng.standard_normal(n) * 10.0 ** rng.uniform(-3, 1.5, n)).astype(np.float32)
    m = (rng.standard_normal(n) * 1e-3).astype(np.float32)
    v = (rng.standard_normal(n) ** 2 * 1e-5 + 1e-7).astype(np.float32)
    grads = [(rng.standard_normal(n) * 1e-2).astype(np.float32) for _ in range(3)]
    for decay, gs, t in ((0.1, 1.0, 1), (0.01, 0.3, 7), (0.5, -0.125, 1000)):
        h = dict(lr=1e-3, decay=decay, beta1=0.9, beta2=0.95, eps=1e-8, step=t, gs=gs)
        w32, m32, v32, *off = ref.step32(ref.mean32(grads), w, m, v, h, bits)
        w64, m64, v64, bw, bm, bv = ref.step64(grads, w, m, v, h, bits)
        for got, want, b in ((w32, w64, bw), (m32, m64, bm), (v32, v64, bv)):
            assert np.all(np.abs(got - want) <= b)
        # and the bound is below a thousandth of the move and a millionth of the weight
        assert np.all(bw <= 1e-3 * np.abs(w64 - w) + 1e-6 * np.abs(w))


@no_device
def test_sumsq_refuses_its_own_workspace():
    """The sum is written: over an entry of the table it would leave addresses
    that the next launch follows."""
    t = _table()
    total = 4 * 128 + 256 + 256 + 2048 * 8  # entries, rank pointers, count, partial sums
    for at in (0, 64, total - 8):
        assert a.zs_grad_sumsq_multi(t, WS + at, stream=0, check=False) == z.ZS_ERR_ALIAS, at
    for at in (-8, total):
        assert a.zs_grad_sumsq_multi(t, WS + at, stream=0, check=False) != z.ZS_ERR_ALIAS, at
