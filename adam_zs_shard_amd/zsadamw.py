"""Thin ctypes binding of libzshard's AdamW operators (include/zsadamw.h), same
names as the C ABI.

Argument marshalling only, as in `zshard`: tensors are used for their device
addresses, plain integers are accepted as addresses too, and there is no CPU
fallback.
"""

from __future__ import annotations

import ctypes as C

from . import zshard as z

ZS_F32 = 3
ZS_STATE8_BLOCK = 256
ZS_ROUND_NEAREST, ZS_ROUND_STOCHASTIC = 0, 1
ZS_STATE8_M, ZS_STATE8_V = 0, 1

DTYPE_NAMES = {**z.DTYPE_NAMES, "f32": ZS_F32}
ROUNDINGS = {"nearest": ZS_ROUND_NEAREST, "stochastic": ZS_ROUND_STOCHASTIC}
KINDS = {"m": ZS_STATE8_M, "v": ZS_STATE8_V}

EXPORTS = [
    "zs_adamw_workspace_bytes", "zs_adamw_upload", "zs_adamw_step_multi", "zs_grad_sumsq_multi",
    "zs_state8_encode", "zs_state8_decode", "zs_adamw_steps_bytes", "zs_adamw_steps_init",
    "zs_adamw_steps_advance", "zs_adamw_steps_status", "zs_adamw_step_multi_dev",
]


class zs_adamw_piece(C.Structure):
    _fields_ = [("len", C.c_int64), ("w", C.c_void_p), ("m", C.c_void_p), ("v", C.c_void_p),
                ("m_scale", C.c_void_p), ("v_scale", C.c_void_p), ("param", C.c_void_p),
                ("g_mean", C.c_void_p), ("grads", C.POINTER(C.c_void_p)),
                ("weight_decay", C.c_double), ("lr_scale", C.c_double), ("index", C.c_int64)]


class zs_adamw_table(C.Structure):
    _fields_ = [("workspace", C.c_void_p), ("nchunks", C.c_int64), ("chunk_elems", C.c_int64),
                ("npieces", C.c_int32), ("p", C.c_int32), ("grad_dtype", C.c_int32),
                ("param_dtype", C.c_int32), ("state_bits", C.c_int32), ("has_mean", C.c_int32),
                ("on_lines", C.c_int32), ("reserved", C.c_int32)]


class zs_adamw_hparams(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double),
                ("eps", C.c_double), ("step", C.c_int64), ("grad_scale", C.c_double),
                ("max_norm", C.c_double), ("seed", C.c_uint64), ("rounding", C.c_int32),
                ("skip_nonfinite", C.c_int32)]


class zs_adamw_steps(C.Structure):
    _fields_ = [("dev", C.c_void_p), ("first_step", C.c_int64), ("nsteps", C.c_int32),
                ("reserved", C.c_int32)]


_lib = None


def lib():
    global _lib
    if _lib is None:
        L = z.lib()
        i32, i64, vp = C.c_int32, C.c_int64, C.c_void_p
        L.zs_adamw_workspace_bytes.argtypes = [C.POINTER(i64), i32, i32]
        L.zs_adamw_workspace_bytes.restype = C.c_size_t
        L.zs_adamw_upload.argtypes = [C.POINTER(zs_adamw_piece), i32, i32, i32, i32, i32, vp,
                                      C.c_size_t, vp, C.POINTER(zs_adamw_table)]
        L.zs_adamw_upload.restype = i32
        L.zs_adamw_step_multi.argtypes = [C.POINTER(zs_adamw_table), C.POINTER(zs_adamw_hparams),
                                          vp, vp]
        L.zs_adamw_step_multi.restype = i32
        L.zs_grad_sumsq_multi.argtypes = [C.POINTER(zs_adamw_table), i32, i32, vp, vp]
        L.zs_grad_sumsq_multi.restype = i32
        L.zs_state8_encode.argtypes = [vp, i64, i32, vp, vp, vp]
        L.zs_state8_encode.restype = i32
        L.zs_state8_decode.argtypes = [vp, vp, i64, i32, vp, vp]
        L.zs_state8_decode.restype = i32
        steps, hp = C.POINTER(zs_adamw_steps), C.POINTER(zs_adamw_hparams)
        L.zs_adamw_steps_bytes.argtypes = [i32]
        L.zs_adamw_steps_bytes.restype = C.c_size_t
        L.zs_adamw_steps_init.argtypes = [hp, C.POINTER(C.c_double), i32, vp, C.c_size_t, vp, steps]
        L.zs_adamw_steps_init.restype = i32
        L.zs_adamw_steps_advance.argtypes = [steps, vp, vp]
        L.zs_adamw_steps_advance.restype = i32
        L.zs_adamw_steps_status.argtypes = [steps, C.POINTER(i64), C.POINTER(i32), vp]
        L.zs_adamw_steps_status.restype = i32
        L.zs_adamw_step_multi_dev.argtypes = [C.POINTER(zs_adamw_table), steps, hp, vp, vp]
        L.zs_adamw_step_multi_dev.restype = i32
        _lib = L
    return _lib


def _named(x, names) -> int:
    return names[x] if x.__class__ is str else int(x or 0)


def hparams(lr, beta1, beta2, eps, step, *, grad_scale=1.0, max_norm=0.0, rounding="stochastic",
            seed=0, skip_nonfinite=False) -> zs_adamw_hparams:
    """rounding: of 8-bit moments, "stochastic" or "nearest"; over a run, v does not follow its
    gradient if it is rounded to nearest.  seed: of the random bits; the step is mixed in, so one
    seed does for a run."""
    return zs_adamw_hparams(float(lr), float(beta1), float(beta2), float(eps), int(step),
                            float(grad_scale), float(max_norm), int(seed) & (2**64 - 1),
                            _named(rounding, ROUNDINGS), int(skip_nonfinite))


def zs_adamw_workspace_bytes(lens, p: int) -> int:
    return lib().zs_adamw_workspace_bytes((C.c_int64 * max(len(lens), 1))(*lens), len(lens), p)


def zs_adamw_upload(pieces, p: int, grad_dtype, param_dtype, state_bits: int, workspace,
                    ws_bytes: int, *, stream=None) -> zs_adamw_table:
    """pieces: [dict(len, grads, w, m, v, m_scale, v_scale, param, g_mean, weight_decay=0,
    lr_scale=1, index=0)] with device addresses (or tensors) at each tensor's first element;
    what the table does not need may be missing.  grad_dtype: "f16", "bf16" or "f32";
    param_dtype: "f16", "bf16" or None; state_bits: 32, 8 or 0 (gradients only)."""
    arr = (zs_adamw_piece * max(len(pieces), 1))()
    keep = []
    for d, q in zip(arr, pieces):
        grads = q["grads"]
        if len(grads) != p:
            raise ValueError(f"{len(grads)} gradients for {p} ranks")
        d.grads, g_keep = z._ptr_array(grads)
        keep.append(g_keep)
        d.len = int(q["len"])
        for name in ("w", "m", "v", "m_scale", "v_scale", "param", "g_mean"):
            setattr(d, name, z._addr(q.get(name)))
        d.weight_decay = float(q.get("weight_decay", 0.0))
        d.lr_scale = float(q.get("lr_scale", 1.0))
        d.index = int(q.get("index", 0))
    table = zs_adamw_table()
    st = lib().zs_adamw_upload(arr, len(pieces), p, _named(grad_dtype, DTYPE_NAMES),
                               _named(param_dtype, z.DTYPE_NAMES), state_bits, z._addr(workspace),
                               ws_bytes, z._stream(stream), C.byref(table))
    del keep
    z._check(st, "zs_adamw_upload")
    return table


def zs_adamw_step_multi(table: zs_adamw_table, hp: zs_adamw_hparams, sumsq=None, *, stream=None,
                        check=True) -> int:
    """sumsq: a float64 device scalar (see zs_grad_sumsq_multi), needed to clip or to skip."""
    st = lib().zs_adamw_step_multi(C.byref(table), C.byref(hp), z._addr(sumsq), z._stream(stream))
    if check:
        z._check(st, "zs_adamw_step_multi")
    return st


def zs_adamw_steps_bytes(nsteps: int) -> int:
    return lib().zs_adamw_steps_bytes(nsteps)


def zs_adamw_steps_init(hp: zs_adamw_hparams, nsteps: int, dev, nbytes: int, *, lrs=None,
                        stream=None) -> zs_adamw_steps:
    """lrs: nsteps learning rates, or None for hp's at every step."""
    if lrs is not None:
        if len(lrs) != nsteps:
            raise ValueError(f"{len(lrs)} learning rates for {nsteps} steps")
        lrs = (C.c_double * max(nsteps, 1))(*lrs)
    t = zs_adamw_steps()
    z._check(lib().zs_adamw_steps_init(C.byref(hp), lrs, nsteps, z._addr(dev), nbytes,
                                       z._stream(stream), C.byref(t)), "zs_adamw_steps_init")
    return t


def zs_adamw_steps_advance(steps: zs_adamw_steps, sumsq=None, *, stream=None, check=True) -> int:
    st = lib().zs_adamw_steps_advance(C.byref(steps), z._addr(sumsq), z._stream(stream))
    if check:
        z._check(st, "zs_adamw_steps_advance")
    return st


def zs_adamw_steps_status(steps: zs_adamw_steps, *, stream=None):
    """(cursor, exhausted) read back from the device."""
    cur, ex = C.c_int64(), C.c_int32()
    z._check(lib().zs_adamw_steps_status(C.byref(steps), C.byref(cur), C.byref(ex),
                                         z._stream(stream)), "zs_adamw_steps_status")
    return cur.value, ex.value


def zs_adamw_step_multi_dev(table: zs_adamw_table, steps: zs_adamw_steps, hp: zs_adamw_hparams,
                            sumsq=None, *, stream=None, check=True) -> int:
    """hp: grad_scale, max_norm, seed, rounding and skip_nonfinite; the rest is the step table's."""
    st = lib().zs_adamw_step_multi_dev(C.byref(table), C.byref(steps), C.byref(hp),
                                       z._addr(sumsq), z._stream(stream))
    if check:
        z._check(st, "zs_adamw_step_multi_dev")
    return st


def zs_grad_sumsq_multi(table: zs_adamw_table, sumsq, *, store_mean=False, accumulate=False,
                        stream=None, check=True) -> int:
    st = lib().zs_grad_sumsq_multi(C.byref(table), int(store_mean), int(accumulate),
                                   z._addr(sumsq), z._stream(stream))
    if check:
        z._check(st, "zs_grad_sumsq_multi")
    return st


def zs_state8_encode(x, n: int, kind, codes, scales, *, stream=None, check=True) -> int:
    """n fp32 moments to codes (n bytes) and scales; kind: "m" or "v"."""
    st = lib().zs_state8_encode(z._addr(x), n, _named(kind, KINDS), z._addr(codes),
                                z._addr(scales), z._stream(stream))
    if check:
        z._check(st, "zs_state8_encode")
    return st


def zs_state8_decode(codes, scales, n: int, kind, x, *, stream=None, check=True) -> int:
    st = lib().zs_state8_decode(z._addr(codes), z._addr(scales), n, _named(kind, KINDS),
                                z._addr(x), z._stream(stream))
    if check:
        z._check(st, "zs_state8_decode")
    return st
