"""Binding of the 8-bit-integer layer operators (include/batchlas.h, "8-bit-integer
layer operators"): argument checks and marshalling only, as in layer.py, whose
conventions on tensors and streams hold here too.

Nothing is recorded for automatic differentiation.  int8_matmul, block_norm and
int8_quant with values refuse floating tensors whose gradient or tangent would be
lost; the norms' gradient is block_norm_grad, and codes have none.

Rows of int8 codes are held in whole 16 bytes: a code tensor [rows, n] is, where n is
not a multiple of 16, a view of the first n columns of a wider one, as int8_quant
and block_norm return it.  What is behind them may hold anything.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd import forward_ad

from . import layer as _layer
from .layer import _TYPES, _float_type, _gpu, _on, _place, _refuse_gradients, _rows, _vector

_I8, _F32 = torch.int8, torch.float32


def _codes(t, name: str):
    """(rows, columns, row stride) of int8 codes, whose rows are read in whole 16 bytes."""
    if t.dtype is not _I8:
        raise TypeError(f"{name} must be torch.int8, not {t.dtype}")
    if t.dim() != 2:
        try:
            t = t.view(-1, t.shape[-1])
        except (RuntimeError, IndexError):
            raise ValueError(f"{name} must be a matrix, or rows of one row stride") from None
    rows, n = t.shape
    ld, step = t.stride()
    if step != 1 and n > 1:
        raise ValueError(f"{name} must have contiguous rows")
    held = (n + 15) // 16 * 16
    if rows <= 1:
        ld = held
    if ld % 16 or t.data_ptr() % 16:
        raise ValueError(f"rows of {name} must start at multiples of 16 bytes")
    if held != n and rows and t.storage_offset() + (rows - 1) * ld + held > t.untyped_storage().nbytes():
        raise ValueError(f"the last row of {name} must be held in whole 16 bytes")
    return rows, n, ld


def _new_codes(x, n: int):
    """Codes of x's shape, [..., n]."""
    held = (n + 15) // 16 * 16
    q = x.new_empty((*x.shape[:-1], held), dtype=_I8)
    return q if held == n else q[..., :n]


def int8_quant(x, *, given=None, values=False, out=None, scales=None, stream=None):
    """Round the rows of x (tokens, or the channels of weights) to 8-bit integers:
    returns (q, scales, values).

    q is int8 of x's shape, within -127..127; scales are float32 [rows], the rows'
    largest magnitudes over 127; a value is its code times its row's scale.
    given: float32 [rows], scales to round under in place of the rows' own (values
    beyond 127 of them saturate).  values=True (or a tensor): also what the codes
    stand for, in x's type; None where not asked for.
    """
    if stream is not None:
        return _on(stream, int8_quant, x, given=given, values=values, out=out, scales=scales)
    lib = _layer._lib or _layer._bind()
    ty = _float_type(x, "x")
    if values is False:
        values = None
    if values is not None:
        _refuse_gradients(x, given)
    at = _gpu(x)
    rows, n, ldx = _rows(x, "x")
    if out is None:
        out = _new_codes(x, n)
    qrows, qn, ldq = _codes(out, "out")
    if qrows != rows or qn != n:
        raise ValueError(f"out must be {rows} x {n}, not {qrows} x {qn}")
    gp = sp = None
    if given is not None:
        if scales is not None:
            raise ValueError("scales are either given or computed")
        gp = _vector(given, "given", _F32, rows)
    else:
        if scales is None:
            scales = x.new_empty(rows, dtype=_F32)
        sp = _vector(scales, "scales", _F32, rows)
    vp, ldv = None, 0
    if values is not None:
        if values is True:
            values = torch.empty_like(x)
        ldv = _rows(values, "values", x.dtype, (rows, n))[2]
        vp = values.data_ptr()
    s = _place(at, (out, given, scales, values))
    st = lib.batchlas_integer_quant(ty, rows, n, x.data_ptr(), ldx, gp, out.data_ptr(), ldq, sp, vp, ldv, s)
    if st:
        _layer._check(st)
    return out, (scales if given is None else given), values


def int8_matmul(x, w, x_scales, w_scales, *, out=None, out_dtype=None, stream=None):
    """y = x W^T for 8-bit integers x [m, k] and w [n, k] with scales for each token and channel.

    x_scales is float32 [m], w_scales float32 [n].  Sums are exact.  y [m, n] is
    `out`, or a new tensor of out_dtype (bfloat16 where None).
    """
    if stream is not None:
        return _on(stream, int8_matmul, x, w, x_scales, w_scales, out=out, out_dtype=out_dtype)
    lib = _layer._lib or _layer._bind()
    if x_scales.requires_grad or w_scales.requires_grad or forward_ad._current_level >= 0:
        _refuse_gradients(x_scales, w_scales)
    at = _gpu(x)
    m, k, ldx = _codes(x, "x")
    n, wk, ldw = _codes(w, "w")
    if wk != k:
        raise ValueError(f"x has {k} columns and w {wk}")
    xs, ws = _vector(x_scales, "x_scales", _F32, m), _vector(w_scales, "w_scales", _F32, n)
    if out is None:
        out_dtype = out_dtype or torch.bfloat16
        out = x.new_empty((*x.shape[:-1], n), dtype=out_dtype)
    yt = _float_type(out, "out")
    ldy = _rows(out, "out", out_dtype, (m, n))[2]
    s = _place(at, (w, x_scales, w_scales, out))
    st = lib.batchlas_integer_matmul(yt, m, n, k, x.data_ptr(), ldx, xs, w.data_ptr(), ldw, ws, out.data_ptr(), ldy, s)
    if st:
        _layer._check(st)
    return out


def _gate(gate, rows: int, n: int, dtype):
    """(pointer, rows, row stride) of a gate: [n], or a row for each of equally long runs of rows."""
    if gate is None:
        return None, 0, 0
    gates, gn, ldg = _rows(gate, "gate", dtype)
    if gn != n or (rows % gates if gates else rows):
        raise ValueError(f"gate must have {n} columns and a number of rows that divides {rows}, not {gates} x {gn}")
    return gate.data_ptr(), gates, ldg


def block_norm(y, residual, weight, post_weight=None, gate=None, *, residual_scale: float = 1.0, eps: float = 1e-6,
               int8: bool = False, out=None, scales=None, residual_out=None, stream=None):
    """From a block's output y and the residual to the next block's input: returns (v, scales, h).

        u = post_weight * y / rms(y)            (u = y without a post_weight)
        h = residual_scale * residual + gate * u
        v = weight * h / rms(h)

    gate: None, [n], or [gates, n], each row for rows / gates consecutive rows.  v has
    y's type, or with int8=True it is codes with float32 scales [rows], as int8_quant
    gives them and int8_matmul takes them (scales is None otherwise).  h has y's
    type; residual_out may be residual or y itself.
    """
    if stream is not None:
        return _on(stream, block_norm, y, residual, weight, post_weight, gate, residual_scale=residual_scale, eps=eps,
                   int8=int8, out=out, scales=scales, residual_out=residual_out)
    lib = _layer._lib or _layer._bind()
    ty = _float_type(y, "y")
    if y.requires_grad or residual.requires_grad or weight.requires_grad or forward_ad._current_level >= 0 \
            or (post_weight is not None and post_weight.requires_grad) or (gate is not None and gate.requires_grad):
        _refuse_gradients(y, residual, weight, post_weight, gate)
    at = _gpu(y)
    rows, n, ldy = _rows(y, "y")
    dt = y.dtype
    ldx = _rows(residual, "residual", dt, (rows, n))[2]
    w = _vector(weight, "weight", dt, n)
    p = _vector(post_weight, "post_weight", dt, n) if post_weight is not None else None
    gp, gates, ldg = _gate(gate, rows, n, dt)
    ldh = n
    if residual_out is None:
        residual_out = residual.new_empty(residual.shape)
    else:
        ldh = _rows(residual_out, "residual_out", dt, (rows, n))[2]
    sp = None
    if int8:
        if out is None:
            out = _new_codes(y, n)
        orows, on, ldv = _codes(out, "out")
        if orows != rows or on != n:
            raise ValueError(f"out must be {rows} x {n}, not {orows} x {on}")
        if scales is None:
            scales = y.new_empty(rows, dtype=_F32)
        sp = _vector(scales, "scales", _F32, rows)
    else:
        if scales is not None:
            raise ValueError("scales are for int8=True")
        ldv = n
        if out is None:
            out = y.new_empty(y.shape)
        else:
            ldv = _rows(out, "out", dt, (rows, n))[2]
    s = _place(at, (residual, weight, post_weight, gate, residual_out, out, scales))
    st = lib.batchlas_block_norm(ty, 1 if int8 else 0, rows, n, y.data_ptr(), ldy, residual.data_ptr(), ldx, w, p, gp,
                                 gates, ldg, residual_scale, eps, residual_out.data_ptr(), ldh, out.data_ptr(), ldv, sp, s)
    if st:
        _layer._check(st)
    return out, scales, residual_out


def block_norm_grad(dv, y, h, weight, post_weight=None, gate=None, dh=None, *, residual_scale: float = 1.0,
                    eps: float = 1e-6, dy=None, dx=None, dgate=None, dweight=None, dpost_weight=None, workspace=None,
                    stream=None):
    """Gradient of block_norm at its stored h: returns (dy, dx, dgate, dweight, dpost_weight).

    dv is the gradient of v (before a rounding to 8 bits), dh the one that reaches h
    on the residual path.  dy and dx (of the residual) have y's type and may each be
    dv, y, h or dh itself, not one another.  dgate has gate's shape and type, or float32 for a gate
    [n]; dweight and dpost_weight are float32 [n].  Each of the three is not computed
    where False is passed, and None where there is no such input.  workspace: a uint8
    tensor of block_norm_grad_workspace(...) bytes, allocated by the call where it is
    None.
    """
    if stream is not None:
        return _on(stream, block_norm_grad, dv, y, h, weight, post_weight, gate, dh, residual_scale=residual_scale,
                   eps=eps, dy=dy, dx=dx, dgate=dgate, dweight=dweight, dpost_weight=dpost_weight, workspace=workspace)
    lib = _layer._lib or _layer._bind()
    ty = _float_type(y, "y")
    at = _gpu(y)
    rows, n, ldy = _rows(y, "y")
    dt = y.dtype
    lddv = _rows(dv, "dv", dt, (rows, n))[2]
    ldh = _rows(h, "h", dt, (rows, n))[2]
    w = _vector(weight, "weight", dt, n)
    p = _vector(post_weight, "post_weight", dt, n) if post_weight is not None else None
    gp, gates, ldg = _gate(gate, rows, n, dt)
    lddh = _rows(dh, "dh", dt, (rows, n))[2] if dh is not None else 0
    lddy = lddx = n
    if dy is None:
        dy = y.new_empty(y.shape)
    else:
        lddy = _rows(dy, "dy", dt, (rows, n))[2]
    if dx is None:
        dx = h.new_empty(h.shape)
    else:
        lddx = _rows(dx, "dx", dt, (rows, n))[2]
    dgp, dgt, lddg = None, 0, 0
    if gate is None:
        if dgate is not None and dgate is not False:
            raise ValueError("dgate needs a gate")
        dgate = None
    elif dgate is False:
        dgate = None
    else:
        lddg = n
        if dgate is None:
            dgate = gate.new_empty(gate.shape, dtype=_F32 if gate.dim() == 1 else dt)
        else:
            if dgate.dtype is not _F32 and dgate.dtype is not dt:
                raise TypeError(f"dgate must be float32 or {dt}, not {dgate.dtype}")
            lddg = _rows(dgate, "dgate", None, (gates, n))[2]
        dgt = 0 if dgate.dtype is _F32 else ty
        dgp = dgate.data_ptr()
    wp = pp = None
    if dweight is None:
        dweight = y.new_empty(n, dtype=_F32)
        wp = dweight.data_ptr()
    elif dweight is False:
        dweight = None
    else:
        wp = _vector(dweight, "dweight", _F32, n)
    if post_weight is None:
        if dpost_weight is not None and dpost_weight is not False:
            raise ValueError("dpost_weight needs a post_weight")
        dpost_weight = None
    elif dpost_weight is None:
        dpost_weight = y.new_empty(n, dtype=_F32)
        pp = dpost_weight.data_ptr()
    elif dpost_weight is False:
        dpost_weight = None
    else:
        pp = _vector(dpost_weight, "dpost_weight", _F32, n)
    kp, size = None, 0
    if workspace is not None:
        size = workspace.numel()
        kp = _vector(workspace, "workspace", torch.uint8, size)
    elif wp or pp or dgp:
        size = block_norm_grad_workspace(dt, rows, n, gates)
        if size:
            workspace = y.new_empty(size, dtype=torch.uint8)
            kp = workspace.data_ptr()
    s = _place(at, (dv, h, weight, post_weight, gate, dh, dy, dx, dgate, dweight, dpost_weight, workspace))
    st = lib.batchlas_block_norm_grad(ty, rows, n, dv.data_ptr(), lddv, y.data_ptr(), ldy, h.data_ptr(), ldh, w, p, gp,
                                      gates, ldg, None if dh is None else dh.data_ptr(), lddh, residual_scale, eps,
                                      dy.data_ptr(), lddy, dx.data_ptr(), lddx, dgt, dgp, lddg, wp, pp, kp, size, s)
    if st:
        _layer._check(st)
    return dy, dx, dgate, dweight, dpost_weight


@functools.lru_cache(maxsize=1024)
def block_norm_grad_workspace(dtype, rows: int, n: int, gates: int = 0) -> int:
    """Bytes of workspace that block_norm_grad of this size needs (host-only); gates: rows of its gate."""
    lib = _layer._lib or _layer._bind()
    size = ctypes.c_int64()
    st = lib.batchlas_block_norm_grad_workspace(_TYPES.get(dtype, -1), rows, n, gates, ctypes.byref(size))
    if st:
        _layer._check(st)
    return size.value
