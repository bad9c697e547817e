"""Thin ctypes binding of libzshard's layer operators (include/zslayer.h), same
names as the C ABI.

Argument marshalling only, as in `zshard`: tensors are used for their device
addresses, types and row strides, plain integers are accepted as addresses too
(then the types are given by name, and rows are contiguous), and there is no CPU
fallback.
"""

from __future__ import annotations

import ctypes as C
import struct

from . import zshard as z
from .zsadamw import DTYPE_NAMES, ZS_F32, _named

ZS_NORM_MAX_COLS = 16384
ZS_NORM_LAYER, ZS_NORM_RMS = 0, 1
ZS_I32, ZS_I64 = 4, 5

KINDS = {"layer": ZS_NORM_LAYER, "rms": ZS_NORM_RMS}
ID_NAMES = {"i32": ZS_I32, "i64": ZS_I64}

EXPORTS = ["zs_norm_forward", "zs_norm_workspace_bytes", "zs_norm_backward", "zs_embed_forward",
           "zs_embed_workspace_bytes", "zs_embed_backward"]


class zs_norm_args(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("kind", C.c_int32), ("dtype", C.c_int32),
                ("w_dtype", C.c_int32), ("reserved", C.c_int32), ("eps", C.c_double),
                ("x", C.c_void_p), ("residual", C.c_void_p), ("total", C.c_void_p),
                ("y", C.c_void_p), ("x_stride", C.c_int64), ("residual_stride", C.c_int64),
                ("total_stride", C.c_int64), ("y_stride", C.c_int64), ("gamma", C.c_void_p),
                ("beta", C.c_void_p), ("mean", C.c_void_p), ("rstd", C.c_void_p),
                ("stream", C.c_void_p)]


class zs_norm_grad_args(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("kind", C.c_int32), ("dtype", C.c_int32),
                ("w_dtype", C.c_int32), ("grad_dtype", C.c_int32), ("accumulate", C.c_int32),
                ("reserved", C.c_int32), ("dy", C.c_void_p), ("x", C.c_void_p),
                ("dres", C.c_void_p), ("dx", C.c_void_p), ("dy_stride", C.c_int64),
                ("x_stride", C.c_int64), ("dres_stride", C.c_int64), ("dx_stride", C.c_int64),
                ("gamma", C.c_void_p), ("mean", C.c_void_p), ("rstd", C.c_void_p),
                ("dgamma", C.c_void_p), ("dbeta", C.c_void_p), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t), ("stream", C.c_void_p)]


class zs_embed_args(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("rows", C.c_int64), ("cols", C.c_int64),
                ("first_row", C.c_int64), ("id_dtype", C.c_int32), ("dtype", C.c_int32),
                ("table_dtype", C.c_int32), ("reserved", C.c_int32), ("scale", C.c_double),
                ("ids", C.c_void_p), ("table", C.c_void_p), ("y", C.c_void_p),
                ("y_stride", C.c_int64), ("pos_ids", C.c_void_p), ("pos_table", C.c_void_p),
                ("pos_rows", C.c_int64), ("stream", C.c_void_p)]


class zs_embed_grad_args(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("rows", C.c_int64), ("cols", C.c_int64),
                ("first_row", C.c_int64), ("id_dtype", C.c_int32), ("dtype", C.c_int32),
                ("grad_dtype", C.c_int32), ("accumulate", C.c_int32), ("scale", C.c_double),
                ("ids", C.c_void_p), ("dy", C.c_void_p), ("dy_stride", C.c_int64),
                ("grad", C.c_void_p), ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t),
                ("stream", C.c_void_p)]


_lib = None


def lib():
    global _lib
    if _lib is None:
        L = z.lib()
        i64 = C.c_int64
        for name, args in (("zs_norm_forward", zs_norm_args), ("zs_norm_backward", zs_norm_grad_args),
                           ("zs_embed_forward", zs_embed_args),
                           ("zs_embed_backward", zs_embed_grad_args)):
            getattr(L, name).argtypes = [C.POINTER(args)]
            getattr(L, name).restype = C.c_int32
        L.zs_norm_workspace_bytes.argtypes = [i64, i64]
        L.zs_norm_workspace_bytes.restype = C.c_size_t
        L.zs_embed_workspace_bytes.argtypes = [i64, i64, i64]
        L.zs_embed_workspace_bytes.restype = C.c_size_t
        _lib = L
    return _lib


# ----------------------------------------------------------------- marshalling
# The argument structs are packed as bytes, which takes 1 us; 3 us as instances of
# the classes above (a launch is 3.4 us).

_CODES = {C.c_int64: "q", C.c_int32: "i", C.c_double: "d", C.c_void_p: "P", C.c_size_t: "N"}
_calls = {}  # name: (the struct's pack, the function on bytes)
_types = {}  # torch's types: zs_dtype or zs_id_dtype
_torch = {}  # and back


def _load(name: str, args):
    import torch

    pack = struct.Struct("".join(_CODES[t] for _, t in args._fields_))
    assert pack.size == C.sizeof(args)
    lib()
    _types.update({torch.float16: z.ZS_F16, torch.bfloat16: z.ZS_BF16, torch.float32: ZS_F32,
                   torch.int32: ZS_I32, torch.int64: ZS_I64})
    _torch.update({code: t for t, code in _types.items()})
    _calls[name] = pack.pack, C.CFUNCTYPE(C.c_int32, C.c_char_p)((name, z.lib()))
    return _calls[name]


def _type(x, given, names) -> int:
    """The type code of an operand: as given, or its tensor's."""
    if given is None and x is not None and x.__class__ is not int:
        return _types.get(x.dtype, 0)
    return _named(given, names)


def _rows(x, cols: int, dtype):
    """(address, stride) of rows of activations of torch's dtype.  A tensor's last dimension
    is a row, and more than two dimensions are rows of one stride."""
    if x is None:
        return 0, cols
    if x.__class__ is int:
        return x, cols
    if x.dtype is not dtype:
        raise ValueError(f"{x.dtype}, {dtype} expected")
    st = x.stride()
    if len(st) == 2:
        stride, step = st
        if step != 1 and x.shape[1] != 1:
            raise ValueError("the elements of a row lie apart")
        return x.data_ptr(), stride if stride >= cols or x.shape[0] > 1 else cols
    if not x.is_contiguous():
        raise ValueError("rows of more than one stride")
    return x.data_ptr(), x.shape[-1] if len(st) > 2 else cols


def _flat(x, dtype):
    """The address of an operand of torch's dtype that has no strides."""
    if x is None:
        return 0
    if x.__class__ is int:
        return x
    if x.dtype is not dtype:
        raise ValueError(f"{x.dtype}, {dtype} expected")
    if not x.is_contiguous():
        raise ValueError("a contiguous tensor expected")
    return x.data_ptr()


# ----------------------------------------------------------------- entry points

def zs_norm_forward(rows: int, cols: int, x, y, gamma=None, beta=None, *, kind="layer", eps=1e-5,
                    residual=None, total=None, mean=None, rstd=None, dtype=None, w_dtype=None,
                    stream=None, check=True) -> int:
    """kind: "layer" or "rms".  With a residual, total gets x + residual, and its norm goes to y.
    dtype: of x, residual, total and y; w_dtype: of gamma and beta; "f16", "bf16" or "f32"."""
    pack, call = _calls.get("zs_norm_forward") or _load("zs_norm_forward", zs_norm_args)
    dt = _type(x, dtype, DTYPE_NAMES)
    w = gamma if gamma is not None else beta
    wdt = _type(w, w_dtype, DTYPE_NAMES) if w is not None else dt
    t, tw, f32 = _torch.get(dt), _torch.get(wdt), _torch[ZS_F32]
    px, sx = _rows(x, cols, t)
    pr, sr = _rows(residual, cols, t)
    pt, st_ = _rows(total, cols, t)
    py, sy = _rows(y, cols, t)
    st = call(pack(rows, cols, _named(kind, KINDS), dt, wdt, 0, eps, px, pr, pt, py, sx, sr, st_, sy,
                   _flat(gamma, tw), _flat(beta, tw), _flat(mean, f32), _flat(rstd, f32),
                   z._stream(stream) or 0))
    if st and check:
        z._check(st, "zs_norm_forward")
    return st


def zs_norm_workspace_bytes(rows: int, cols: int) -> int:
    return lib().zs_norm_workspace_bytes(rows, cols)


def zs_norm_backward(rows: int, cols: int, dy, x, rstd, dx, *, mean=None, gamma=None, dres=None,
                     dgamma=None, dbeta=None, kind="layer", accumulate=False, workspace=None,
                     ws_bytes=0, dtype=None, w_dtype=None, grad_dtype=None, stream=None,
                     check=True) -> int:
    """x: what the forward pass normalised (its total where it had a residual), mean and rstd what
    it left.  dres: a gradient that is added to dx.  accumulate: dgamma and dbeta are added to."""
    pack, call = _calls.get("zs_norm_backward") or _load("zs_norm_backward", zs_norm_grad_args)
    dt = _type(x, dtype, DTYPE_NAMES)
    wdt = _type(gamma, w_dtype, DTYPE_NAMES) if gamma is not None else dt
    g = dgamma if dgamma is not None else dbeta
    gdt = _type(g, grad_dtype, DTYPE_NAMES) if g is not None else dt
    t, tg, f32 = _torch.get(dt), _torch.get(gdt), _torch[ZS_F32]
    pd, sd = _rows(dy, cols, t)
    px, sx = _rows(x, cols, t)
    pr, sr = _rows(dres, cols, t)
    po, so = _rows(dx, cols, t)
    st = call(pack(rows, cols, _named(kind, KINDS), dt, wdt, gdt, int(accumulate), 0, pd, px, pr, po, sd, sx,
                   sr, so, _flat(gamma, _torch.get(wdt)), _flat(mean, f32), _flat(rstd, f32),
                   _flat(dgamma, tg), _flat(dbeta, tg), z._addr(workspace) or 0, ws_bytes,
                   z._stream(stream) or 0))
    if st and check:
        z._check(st, "zs_norm_backward")
    return st


def zs_embed_forward(tokens: int, ids, rows: int, cols: int, table, y, *, scale=1.0, first_row=0,
                     pos_ids=None, pos_rows=0, pos_table=None, dtype=None, table_dtype=None,
                     id_dtype=None, stream=None, check=True) -> int:
    """dtype: of y; table_dtype: of table and pos_table; id_dtype: of ids and pos_ids, "i32" or
    "i64".  Ids outside first_row .. first_row + rows - 1 give zeros."""
    pack, call = _calls.get("zs_embed_forward") or _load("zs_embed_forward", zs_embed_args)
    dt, tdt, idt = (_type(y, dtype, DTYPE_NAMES), _type(table, table_dtype, DTYPE_NAMES),
                    _type(ids, id_dtype, ID_NAMES))
    ti, tt = _torch.get(idt), _torch.get(tdt)
    py, sy = _rows(y, cols, _torch.get(dt))
    st = call(pack(tokens, rows, cols, first_row, idt, dt, tdt, 0, scale, _flat(ids, ti),
                   _flat(table, tt), py, sy, _flat(pos_ids, ti), _flat(pos_table, tt), pos_rows,
                   z._stream(stream) or 0))
    if st and check:
        z._check(st, "zs_embed_forward")
    return st


def zs_embed_workspace_bytes(tokens: int, rows: int, cols: int) -> int:
    return lib().zs_embed_workspace_bytes(tokens, rows, cols)


def zs_embed_backward(tokens: int, ids, rows: int, cols: int, dy, grad, workspace=None, ws_bytes=0, *,
                      scale=1.0, first_row=0, accumulate=False, dtype=None, grad_dtype=None,
                      id_dtype=None, stream=None, check=True) -> int:
    """accumulate: grad's rows that a token names are added to; else all of grad is written."""
    pack, call = _calls.get("zs_embed_backward") or _load("zs_embed_backward", zs_embed_grad_args)
    dt, gdt, idt = (_type(dy, dtype, DTYPE_NAMES), _type(grad, grad_dtype, DTYPE_NAMES),
                    _type(ids, id_dtype, ID_NAMES))
    pd, sd = _rows(dy, cols, _torch.get(dt))
    st = call(pack(tokens, rows, cols, first_row, idt, dt, gdt, int(accumulate), scale,
                   _flat(ids, _torch.get(idt)), pd, sd, _flat(grad, _torch.get(gdt)),
                   z._addr(workspace) or 0, ws_bytes, z._stream(stream) or 0))
    if st and check:
        z._check(st, "zs_embed_backward")
    return st
