"""Host-side tests of the layer operators' C ABI (no GPU, no kernel launched):
symbols, sizes, and the refusal of every bad argument before anything reaches the
device; and the 64-bit references that the GPU tests use, against torch's
gradients and against differences."""

import ctypes as C
import os
import re

import pytest
import torch

import layer_diff
import layer_ref as ref
from adam_zs_shard_amd import zshard as z
from adam_zs_shard_amd import zslayer as a

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "zslayer.h")
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: CPU-only test")
FAKE = 1 << 40


def at(i):
    """A fake address, 16 GiB from the next."""
    return FAKE + (i << 34)


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(zs_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(a.EXPORTS)
    for n in names:
        assert hasattr(a.lib(), n), n


def test_structs_match_the_header(tmp_path):
    """Sizes and offsets as the C compiler has them."""
    import subprocess

    src = tmp_path / "offsets.c"
    rows = []
    for s in ("zs_norm_args", "zs_norm_grad_args", "zs_embed_args", "zs_embed_grad_args"):
        rows.append(f'printf("{s} %zu\\n", sizeof({s}));')
        for f, _ in getattr(a, s)._fields_:
            rows.append(f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));')
    src.write_text('#include <stdio.h>\n#include "zslayer.h"\nint main(void) {' + "\n".join(rows)
                   + "return 0; }")
    exe = tmp_path / "offsets"
    subprocess.run(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n"):
        if not line:
            continue
        name, n = line.split()
        s, _, f = name.partition(".")
        got = getattr(getattr(a, s), f).offset if f else C.sizeof(getattr(a, s))
        assert got == int(n), name


# ----------------------------------------------------------------- the norm

def norm(rows=4, cols=100, check=False, **k):
    k = {**dict(x=at(0), y=at(1), gamma=at(2), beta=at(3), residual=at(4), total=at(5), mean=at(6),
                rstd=at(7), dtype="bf16", w_dtype="bf16"), **k}
    return a.zs_norm_forward(rows, cols, k.pop("x"), k.pop("y"), k.pop("gamma"), k.pop("beta"),
                             stream=0, check=check, **k)


@no_device
def test_norm_refuses():
    assert norm(rows=-1) == z.ZS_ERR_ARG and norm(cols=0) == z.ZS_ERR_ARG
    assert norm(kind=2) == z.ZS_ERR_ARG
    assert norm(cols=a.ZS_NORM_MAX_COLS + 1) == z.ZS_ERR_RANGE
    assert norm(rows=1 << 58) == z.ZS_ERR_RANGE
    for eps in (-1e-5, float("inf"), float("nan")):
        assert norm(eps=eps) == z.ZS_ERR_ARG
    assert norm(dtype=0) == z.ZS_ERR_DTYPE and norm(dtype=4) == z.ZS_ERR_DTYPE
    assert norm(w_dtype=7) == z.ZS_ERR_DTYPE
    for name in ("x", "y", "total"):
        assert norm(**{name: None}) == z.ZS_ERR_NULL, name
    for name in ("x", "y", "total", "residual", "gamma", "beta"):
        assert norm(**{name: at(9) + 1}) == z.ZS_ERR_ARG, name
    for name in ("mean", "rstd"):
        assert norm(**{name: at(9) + 2}) == z.ZS_ERR_ARG, name
    # no rows: nothing to do, nothing looked at
    assert norm(rows=0, x=None, y=None) == z.ZS_OK
    with pytest.raises(z.ZsError):
        norm(cols=0, check=True)


# doubles whose nearest fp32 is infinite; 3.4028235e38 still is the largest finite one
BEYOND_F32 = [1e39, 3.5e38, 1e300]
LARGEST_F32 = 3.4028235e38


@no_device
def test_refuses_what_fp32_does_not_hold():
    for v in BEYOND_F32:
        assert norm(eps=v) == z.ZS_ERR_ARG
        for x in (v, -v):
            assert embed(scale=x) == z.ZS_ERR_ARG
            assert embed_grad(scale=x) == z.ZS_ERR_ARG
    # what it holds gets as far as the operands
    assert norm(eps=LARGEST_F32, x=None) == z.ZS_ERR_NULL
    for x in (LARGEST_F32, -LARGEST_F32):
        assert embed(scale=x, ids=None) == z.ZS_ERR_NULL
        assert embed_grad(scale=x, dy=None) == z.ZS_ERR_NULL


@no_device
def test_norm_refuses_overlap():
    size = (3 * 100 + 100) * 2
    for over in (dict(y=at(0) + size - 2), dict(total=at(1) + 2), dict(y=at(2) - size + 2), dict(y=at(3)),
                 dict(mean=at(0) + 4), dict(rstd=at(6) + 12), dict(mean=at(1) + size - 4), dict(rstd=at(2)),
                 dict(y=at(5)),                   # both outputs
                 dict(rows=1, y=at(2)),           # of one row: as large as a weight
                 dict(y=at(0) + 200),             # one row on
                 dict(y=at(4) + 2)):
        assert norm(**over) == z.ZS_ERR_ALIAS, over


def _strided(rows, cols, **k):
    """The C call itself, with strides."""
    q = a.zs_norm_args(rows, cols, 0, z.ZS_BF16, z.ZS_BF16, 0, 1e-5, at(0), None, None, at(1), cols, 0, 0,
                       cols, None, None, None, None, None)
    for name, x in k.items():
        setattr(q, name, x)
    return a.lib().zs_norm_forward(q)


@no_device
def test_norm_refuses_strides():
    assert a.lib().zs_norm_forward(None) == z.ZS_ERR_NULL
    assert _strided(4, 100, x_stride=99) == z.ZS_ERR_ARG
    assert _strided(4, 100, y_stride=0) == z.ZS_ERR_ARG
    assert _strided(4, 100, y_stride=-100) == z.ZS_ERR_ARG
    assert _strided(4, 100, x_stride=1 << 60) == z.ZS_ERR_RANGE
    assert _strided(4, 100, reserved=1) == z.ZS_ERR_ARG
    # columns of one wider buffer that meet in the middle, or round the end of a row
    assert _strided(4, 100, x_stride=200, y=at(0) + 198, y_stride=200) == z.ZS_ERR_ALIAS
    assert _strided(4, 100, x_stride=200, y=at(0) + 202, y_stride=200) == z.ZS_ERR_ALIAS
    assert _strided(4, 100, x_stride=200, x=at(0) + 200, y=at(0) + 2, y_stride=200) == z.ZS_ERR_ALIAS
    # the same first row, other rows apart
    assert _strided(4, 100, x_stride=200, y=at(0), y_stride=202) == z.ZS_ERR_ALIAS


def norm_grad(rows=4, cols=100, **k):
    k = {**dict(dy=at(0), x=at(1), rstd=at(2), dx=at(3), mean=at(4), gamma=at(5), dres=at(6), dgamma=at(7),
                dbeta=at(8), workspace=at(9), ws_bytes=1 << 30, dtype="bf16", w_dtype="bf16",
                grad_dtype="f32"), **k}
    return a.zs_norm_backward(rows, cols, k.pop("dy"), k.pop("x"), k.pop("rstd"), k.pop("dx"), stream=0,
                              check=False, **k)


@no_device
def test_norm_grad_refuses():
    assert a.lib().zs_norm_backward(None) == z.ZS_ERR_NULL
    assert norm_grad(rows=-1) == z.ZS_ERR_ARG and norm_grad(kind=5) == z.ZS_ERR_ARG
    assert norm_grad(cols=a.ZS_NORM_MAX_COLS + 1) == z.ZS_ERR_RANGE
    assert norm_grad(accumulate=2) == z.ZS_ERR_ARG
    for name in ("dtype", "w_dtype", "grad_dtype"):
        assert norm_grad(**{name: 9}) == z.ZS_ERR_DTYPE, name
    for name in ("dy", "x", "dx", "mean", "rstd", "workspace"):
        assert norm_grad(**{name: None}) == z.ZS_ERR_NULL, name
    for name in ("dy", "x", "dx", "mean", "rstd", "gamma", "dgamma", "dbeta", "dres"):
        assert norm_grad(**{name: at(11) + 1}) == z.ZS_ERR_ARG, name
    assert norm_grad(workspace=at(9) + 128) == z.ZS_ERR_CAPACITY
    need = a.zs_norm_workspace_bytes(4, 100)
    assert need > 0 and norm_grad(ws_bytes=need - 1) == z.ZS_ERR_CAPACITY
    size = 400 * 2
    for over in (dict(dx=at(1) + 2), dict(dx=at(0) + 200), dict(dgamma=at(8) + 396), dict(dbeta=at(5)),
                 dict(dgamma=at(3) + size - 4), dict(workspace=at(1)), dict(workspace=at(7)),
                 dict(dx=at(9) + need - 2), dict(dgamma=at(2) + 12), dict(dbeta=at(4))):
        assert norm_grad(**over) == z.ZS_ERR_ALIAS, over
    assert norm_grad(rows=0, dgamma=None, dbeta=None, workspace=None) == z.ZS_OK
    assert norm_grad(rows=0, accumulate=True) == z.ZS_OK


def test_workspace_bytes():
    need = a.zs_norm_workspace_bytes
    assert need(1, 1) > 0 and need(1 << 20, 4096) < 64 << 20
    assert need(-1, 5) == 0 and need(5, 0) == 0 and need(5, a.ZS_NORM_MAX_COLS + 1) == 0
    need = a.zs_embed_workspace_bytes
    assert need(0, 1, 1) > 0 and need(1000, 100, 64) >= 1000 * 16
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), ((1 << 28) + 1, 1, 1), (1, (1 << 30) + 1, 1),
                (1, 1, (1 << 20) + 1)):
        assert need(*bad) == 0


# ----------------------------------------------------------------- the table

def embed(tokens=10, rows=50, cols=100, check=False, **k):
    k = {**dict(ids=at(0), table=at(1), y=at(2), pos_ids=at(3), pos_table=at(4), pos_rows=7, dtype="bf16",
                table_dtype="f32", id_dtype="i64"), **k}
    return a.zs_embed_forward(tokens, k.pop("ids"), rows, cols, k.pop("table"), k.pop("y"), stream=0,
                              check=check, **k)


@no_device
def test_embed_refuses():
    assert a.lib().zs_embed_forward(None) == z.ZS_ERR_NULL
    for bad in (dict(tokens=-1), dict(rows=0), dict(cols=0), dict(first_row=-1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(pos_rows=0)):
        assert embed(**bad) == z.ZS_ERR_ARG, bad
    for bad in (dict(tokens=(1 << 28) + 1), dict(rows=(1 << 30) + 1), dict(cols=(1 << 20) + 1),
                dict(pos_rows=(1 << 30) + 1)):
        assert embed(**bad) == z.ZS_ERR_RANGE, bad
    for bad in (dict(dtype=0), dict(table_dtype=4), dict(id_dtype=3), dict(id_dtype=0)):
        assert embed(**bad) == z.ZS_ERR_DTYPE, bad
    for name in ("ids", "table", "y", "pos_ids"):
        assert embed(**{name: None}) == z.ZS_ERR_NULL, name
    for name, off in (("ids", 4), ("table", 2), ("y", 1), ("pos_ids", 4), ("pos_table", 2)):
        assert embed(**{name: at(9) + off}) == z.ZS_ERR_ARG, name
    for over in (dict(y=at(0)), dict(y=at(1) + 50 * 400 - 4), dict(y=at(3) - 1998), dict(y=at(4))):
        assert embed(**over) == z.ZS_ERR_ALIAS, over
    assert embed(tokens=0, ids=None, y=None) == z.ZS_OK
    with pytest.raises(z.ZsError):
        embed(rows=0, check=True)


def embed_grad(tokens=10, rows=50, cols=100, **k):
    k = {**dict(ids=at(0), dy=at(1), grad=at(2), workspace=at(3), ws_bytes=1 << 30, dtype="bf16",
                grad_dtype="f32", id_dtype="i32"), **k}
    return a.zs_embed_backward(tokens, k.pop("ids"), rows, cols, k.pop("dy"), k.pop("grad"), stream=0,
                               check=False, **k)


@no_device
def test_embed_grad_refuses():
    assert a.lib().zs_embed_backward(None) == z.ZS_ERR_NULL
    for bad in (dict(tokens=-1), dict(rows=0), dict(cols=0), dict(first_row=-1), dict(scale=float("nan")),
                dict(accumulate=2)):
        assert embed_grad(**bad) == z.ZS_ERR_ARG, bad
    for bad in (dict(tokens=(1 << 28) + 1), dict(rows=(1 << 30) + 1), dict(cols=(1 << 20) + 1)):
        assert embed_grad(**bad) == z.ZS_ERR_RANGE, bad
    for bad in (dict(dtype=0), dict(grad_dtype=4), dict(id_dtype=3)):
        assert embed_grad(**bad) == z.ZS_ERR_DTYPE, bad
    for name in ("ids", "dy", "grad", "workspace"):
        assert embed_grad(**{name: None}) == z.ZS_ERR_NULL, name
    for name, off in (("ids", 2), ("dy", 1), ("grad", 2)):
        assert embed_grad(**{name: at(9) + off}) == z.ZS_ERR_ARG, name
    need = a.zs_embed_workspace_bytes(10, 50, 100)
    assert embed_grad(ws_bytes=need - 1) == z.ZS_ERR_CAPACITY
    assert embed_grad(workspace=at(3) + 8) == z.ZS_ERR_CAPACITY
    for over in (dict(grad=at(0) + 36), dict(grad=at(1)), dict(workspace=at(2) + 49 * 400 + 256 - 49 * 400 % 256),
                 dict(workspace=at(0)), dict(workspace=at(1))):
        assert embed_grad(**over) == z.ZS_ERR_ALIAS, over
    assert embed_grad(tokens=0, accumulate=True, ids=None, dy=None, workspace=None) == z.ZS_OK


def test_binding_refuses_tensors_that_it_cannot_name():
    x = torch.zeros(4, 20, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        a.zs_norm_forward(4, 10, x[:, ::2], x)
    with pytest.raises(ValueError):
        a.zs_norm_forward(4, 20, x, x, x[:, 0])
    with pytest.raises(ValueError):
        a.zs_embed_forward(4, torch.zeros(8, dtype=torch.int64)[::2], 4, 20, x, x)
    with pytest.raises(ValueError):
        a.zs_norm_forward(4, 10, torch.zeros(2, 2, 20)[:, :, :10], x)
    assert a._rows(x[:, :10], 10, x.dtype) == (x.data_ptr(), 20)
    assert a._rows(x[:1], 20, x.dtype) == (x.data_ptr(), 20)
    assert a._rows(torch.zeros(2, 3, 7), 7, torch.float32)[1] == 7
    # types that do not go together
    f, w, i = torch.zeros(4, 20), torch.zeros(20), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: a.zs_norm_forward(4, 20, x, f), lambda: a.zs_norm_forward(4, 20, f, x),
                 lambda: a.zs_norm_forward(4, 20, f, f, w, w.half()),
                 lambda: a.zs_norm_forward(4, 20, x, x.clone(), rstd=x[0]),
                 lambda: a.zs_norm_backward(4, 20, f, x, w, x),
                 lambda: a.zs_norm_backward(4, 20, f, f, w, f, dgamma=w, dbeta=x[0]),
                 lambda: a.zs_embed_forward(4, i, 4, 20, x, f, pos_ids=i.int(), pos_rows=4, pos_table=x),
                 lambda: a.zs_embed_forward(4, i, 4, 20, x, f, pos_ids=i, pos_rows=4, pos_table=f),
                 lambda: a.zs_embed_backward(4, i, 4, 20, f.double(), f, f, 0)):
        with pytest.raises((ValueError, z.ZsError)):
            call()


# batches around 2^23 elements (where the windows get longer), 16384 tokens (more launches) and
# multiples of 262144 (where the tiles get longer)
@pytest.mark.parametrize("cols", [1, 24, 32, 768, 1000, 4096, 1 << 20])
def test_workspace_of_a_long_batch_does_for_shorter_ones(cols):
    few, tiles = (1 << 23) // cols, 256 * 1024
    ends = [1, few // 2, few, 3 * few // 2, 2 * few, 10_000, 16_384, 20_000, tiles, 2 * tiles, 3 * tiles,
            few // tiles * tiles, 1_000_000, 1 << 28]
    tokens = sorted({t + d for t in ends for d in (-1, 0, 1) if 1 <= t + d <= 1 << 28})
    sizes = [a.zs_embed_workspace_bytes(t, 50257, cols) for t in tokens]
    assert sizes == sorted(sizes)
    # no smaller than what a call of any of them asks for; the workspace lies on the ids, which is seen later
    for i, t in enumerate(tokens):
        for size in {sizes[i], sizes[-1]}:
            q = a.zs_embed_grad_args(t, 5, cols, 0, a.ZS_I64, z.ZS_BF16, z.ZS_BF16, 0, 1.0, 1 << 50, 1 << 52, cols,
                                     1 << 40, 1 << 50, size, None)
            assert a.lib().zs_embed_backward(q) == z.ZS_ERR_ALIAS, (t, size)


# ----------------------------------------------------------------- the references

def _inputs(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return n(rows, cols) * 2 + 0.5, 1 + 0.3 * n(cols), n(cols), n(rows, cols)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_reference_against_autograd_and_differences(kind):
    x, gamma, beta, dy = _inputs(5, 33, 1)
    eps = 1e-5

    def forward(x, gamma, beta):
        m = x.mean(1, keepdim=True) if kind == "layer" else 0.0
        v = ((x - m) ** 2).mean(1, keepdim=True)
        return (x - m) / torch.sqrt(v + eps) * gamma + beta

    out = ref.norm(x, gamma, beta, kind, eps, torch.float32)
    assert torch.allclose(out["y"][0], forward(x, gamma, beta), rtol=1e-12, atol=1e-12)
    if kind == "layer":
        assert torch.allclose(out["y"][0], torch.nn.functional.layer_norm(x, (33,), gamma, beta, eps),
                              rtol=1e-12, atol=1e-12)
    leaves = [t.clone().requires_grad_() for t in (x, gamma, beta)]
    (forward(*leaves) * dy).sum().backward()
    mean = x.mean(1)
    got = ref.norm_grad(dy, x, mean, out["rstd"][0], gamma, torch.zeros_like(x), kind, torch.float32,
                        torch.float32, torch.zeros(33), torch.zeros(33))
    for name, leaf in zip(("dx", "dgamma", "dbeta"), leaves):
        assert torch.allclose(got[name][0], leaf.grad, rtol=1e-10, atol=1e-12), name
    # central differences along a direction: off by a sixth of h^2 times a third derivative
    h = 1e-5
    for i, name in enumerate(("dx", "dgamma", "dbeta")):
        d = torch.randn(leaves[i].shape, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
        args = [x, gamma, beta]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * d, args[i] - h * d
        diff = ((forward(*up) - forward(*down)) * dy).sum() / (2 * h)
        assert abs(diff - (got[name][0] * d).sum()) < 1e-7 * (1 + abs(diff)), name


def _gradients(x, dy, gamma, kind, eps, leave_out=()):
    """The formulas in 64 bits, rounded to fp32, less some of their terms."""
    x, dy, gamma = x.double(), dy.double(), gamma.double()
    u = x - x.mean(1, keepdim=True) if kind == "layer" else x
    r = (u.square().mean(1, keepdim=True) + eps).rsqrt()
    a, h = dy * gamma, u * r
    dx = a - h * (a * h).mean(1, keepdim=True) * ("c2" not in leave_out)
    if kind == "layer" and "c1" not in leave_out:
        dx = dx - a.mean(1, keepdim=True)
    return [t.float() for t in (dx * r, (dy * h).sum(0), dy.sum(0))]


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_differences_tell_wrong_gradients(kind):
    eps = 1e-5
    x, dy, gamma, beta = layer_diff.inputs(40, 768, 808)

    def forward(x, gamma, beta):
        return ref.norm(x.double(), gamma.double(), beta.double(), kind, eps, torch.float32)["y"][0].float()

    dx, dg, db = _gradients(x, dy, gamma, kind, eps)
    layer_diff.check(forward, x, dy, gamma, beta, kind, eps, dx, dg, db)
    one_row = dx.clone()
    one_row[17] = 0
    wrong = [(0 * dx, dg, db), (-dx, dg, db), (1.03 * dx, dg, db), (one_row, dg, db),
             (_gradients(x, dy, gamma, kind, eps, ["c2"])[0], dg, db), (dx, 1.03 * dg, db), (dx, -dg, db),
             (dx, dg, 0 * db), (dx, dg, 1.03 * db), (dx, db, dg)]
    if kind == "layer":
        wrong.append((_gradients(x, dy, gamma, kind, eps, ["c1"])[0], dg, db))
    for got in wrong:
        with pytest.raises(AssertionError):
            layer_diff.check(forward, x, dy, gamma, beta, kind, eps, *got)


def test_embed_reference_against_autograd():
    g = torch.Generator().manual_seed(3)
    table = torch.randn(7, 5, generator=g, dtype=torch.float64, requires_grad=True)
    ids = torch.tensor([3, 3, 0, 6, 3, 1, 0])
    dy = torch.randn(7, 5, generator=g, dtype=torch.float64)
    (torch.nn.functional.embedding(ids, table) * 1.5 * dy).sum().backward()
    got, bound, count = ref.embed_grad(dy, ids, 7, 1.5, torch.zeros(7, 5, dtype=torch.float64), torch.float32)
    assert torch.allclose(got, table.grad, rtol=1e-12) and count.tolist() == [2, 1, 0, 3, 0, 0, 1]
    assert (bound > 0).all()
