"""Binding of the low-bit layer operators (include/batchlas.h, "Low-bit layer
operators"): argument checks and marshalling only, as in the package's other
entry points.  Tensors here are row-major, [rows, columns], with any row stride.

Every operator runs on the current stream, or on `stream`, and tensors that it
allocates (outputs, workspaces) belong to the stream that it runs on.

Nothing is recorded for automatic differentiation.  rmsnorm_quant and
weight_matvec refuse floating tensors whose gradient or tangent would be lost;
the norm's gradient is rmsnorm_grad, and a rounding has none.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd import forward_ad

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3}
_FORMATS = {"int4": 0, "fp4": 1}
_WHOLE_ROWS = 16                # added to a format
_SCALES = {"row": 1, "block": 2}
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu

_lib = _check = None


def _bind():
    """The loaded library (once) and the status check."""
    global _lib, _check
    if _lib is None:
        from . import _check as check, load_library
        _lib, _check = load_library(), check
    return _lib


def _rows(t, name: str, dtype=None, shape=None):
    """(rows, columns, row stride) of a tensor, taken as a matrix of its last dimension."""
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    size = t.shape
    if len(size) == 2:
        rows, n = size
        ld, step = t.stride()
        if step != 1 and n > 1:
            raise ValueError(f"{name} must have contiguous rows")
        if rows <= 1:
            ld = n
    else:
        if not size or not t.is_contiguous():
            raise ValueError(f"{name} must be a matrix, or contiguous")
        n = ld = size[-1]
        rows = t.numel() // n if n else 0
    if shape is not None and (shape[0] != rows or shape[1] != n):
        raise ValueError(f"{name} must be {shape[0]} x {shape[1]}, not {rows} x {n}")
    return rows, n, ld


def _vector(t, name: str, dtype, n: int) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements")
    return t.data_ptr()


def _gpu(t) -> int:
    """The index of the GPU that t is on."""
    at = t.get_device()
    if at < 0:
        raise ValueError("tensors must live on the GPU")
    return at


def _on(stream, operator, *args, **kwargs):
    """The operator with `stream` as the current one, so that what it allocates belongs to it."""
    with torch.cuda.stream(stream):
        return operator(*args, **kwargs)


def _place(at: int, others) -> int:
    """The current stream's handle, after checking that every tensor is on the current device, `at`."""
    for o in others:
        if o is not None and o.get_device() != at:
            raise ValueError("tensors must live on the GPU, on one device")
    if at != torch._C._cuda_getDevice():
        raise ValueError("tensors must live on the current device")
    return torch._C._cuda_getCurrentRawStream(at)


def _float_type(t, name: str) -> int:
    code = _TYPES.get(t.dtype, 3)
    if code == 3:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    return code


def _refuse_gradients(*tensors):
    """Refuses tensors whose gradient, or tangent, the call would lose."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("the gradient would be lost: detach the tensors, or call under torch.no_grad()")
    if forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError("the tangent would be lost, as a gradient would: pass the primal tensors")


def rmsnorm_quant(x, weight, residual=None, *, eps: float = 1e-6, scale: str = "block", out=None,
                  scales=None, residual_out=None, stream=None):
    """Root-mean-square norm of h = x + residual with an output in 8 bits.

    Returns (q, scales, h): q in float8_e4m3fn, of x's shape; scales in
    float8_e8m0fnu [rows, ceil(n / 32)] (scale="block") or float32 [rows]
    (scale="row"); h = x + residual in x's type (None without a residual).
    residual_out may be x or residual itself.
    """
    if stream is not None:
        return _on(stream, rmsnorm_quant, x, weight, residual, eps=eps, scale=scale, out=out,
                   scales=scales, residual_out=residual_out)
    lib = _lib or _bind()
    ty = _float_type(x, "x")
    if x.requires_grad or weight.requires_grad or (residual is not None and residual.requires_grad) \
            or forward_ad._current_level >= 0:
        _refuse_gradients(x, weight, residual)
    at = _gpu(x)
    rows, n, ldx = _rows(x, "x")
    dt = x.dtype
    w = _vector(weight, "weight", dt, n)
    if scale not in _SCALES:
        raise ValueError('scale must be "block" or "row"')
    rp = hp = None
    ldr = ldh = 0
    if residual is not None:
        ldr = _rows(residual, "residual", dt, (rows, n))[2]
        if residual_out is None:
            residual_out = torch.empty_like(x)
        ldh = _rows(residual_out, "residual_out", dt, (rows, n))[2]
        rp, hp = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if out is None:
        out = torch.empty_like(x, dtype=_E4M3)
    ldq = _rows(out, "out", _E4M3, (rows, n))[2]
    lds = 0
    if scale == "block":
        blocks = (n + 31) // 32
        if scales is None:
            scales = x.new_empty((rows, blocks), dtype=_E8M0)
        lds = _rows(scales, "scales", _E8M0, (rows, blocks))[2]
    else:
        if scales is None:
            scales = x.new_empty(rows, dtype=torch.float32)
        _vector(scales, "scales", torch.float32, rows)
    s = _place(at, (weight, residual, residual_out, out, scales))
    st = lib.batchlas_rmsnorm_quant(ty, _SCALES[scale], rows, n, x.data_ptr(), ldx, rp, ldr, w, eps,
                                    hp, ldh, out.data_ptr(), ldq, scales.data_ptr(), lds, s)
    if st:
        _check(st)
    return out, scales, residual_out


def rmsnorm_grad(dy, h, weight, dh=None, *, eps: float = 1e-6, dx=None, dweight=None, workspace=None,
                 stream=None):
    """Gradient of the norm at h: returns (dx, dweight).

    dy is the gradient of the norm's output (before its rounding to 8 bits), dh
    the one that reaches h on the residual path.  dx, in h's type, is the
    gradient of x and of the residual; dweight is float32 [n].  dx may be dy, h
    or dh itself.  dweight=False: not computed.  workspace: a uint8 tensor of
    rmsnorm_grad_workspace(...) bytes, allocated by the call where it is None.
    """
    if stream is not None:
        return _on(stream, rmsnorm_grad, dy, h, weight, dh, eps=eps, dx=dx, dweight=dweight, workspace=workspace)
    lib = _lib or _bind()
    ty = _float_type(h, "h")
    at = _gpu(h)
    rows, n, ldh = _rows(h, "h")
    dt = h.dtype
    lddy = _rows(dy, "dy", dt, (rows, n))[2]
    w = _vector(weight, "weight", dt, n)
    lddh = _rows(dh, "dh", dt, (rows, n))[2] if dh is not None else 0
    if dx is None:
        dx = torch.empty_like(h)
    lddx = _rows(dx, "dx", dt, (rows, n))[2]
    wp = dp = None
    size = 0
    if dweight is not False:
        if dweight is None:
            dweight = h.new_empty(n, dtype=torch.float32)
        dp = _vector(dweight, "dweight", torch.float32, n)
        if workspace is None:
            size = rmsnorm_grad_workspace(h.dtype, rows, n)
            workspace = h.new_empty(size, dtype=torch.uint8) if size else None
        if workspace is not None:
            size = workspace.numel()
            wp = _vector(workspace, "workspace", torch.uint8, size)
    s = _place(at, (dy, weight, dh, dx, dweight if dp else None, workspace if wp else None))
    st = lib.batchlas_rmsnorm_grad(ty, rows, n, dy.data_ptr(), lddy, h.data_ptr(), ldh, w,
                                   None if dh is None else dh.data_ptr(), lddh, eps, dx.data_ptr(), lddx,
                                   dp, wp, size, s)
    if st:
        _check(st)
    return dx, (dweight if dp else None)


@functools.lru_cache(maxsize=1024)
def rmsnorm_grad_workspace(dtype, rows: int, n: int) -> int:
    """Bytes of workspace that rmsnorm_grad of this size needs (host-only)."""
    lib = _lib or _bind()
    size = ctypes.c_int64()
    st = lib.batchlas_rmsnorm_grad_workspace(_TYPES.get(dtype, -1), rows, n, ctypes.byref(size))
    if st:
        _check(st)
    return size.value


def _codes(codes, k: int):
    """(rows, row stride) of codes; a row is read in whole 16 bytes, so it has to hold them."""
    n, width, ldc = _rows(codes, "codes", torch.uint8)
    need = (k + 31) // 32 * 16
    if codes.dim() != 2 or width < need:
        raise ValueError(f"codes must be rows of at least {need} bytes")
    return n, (ldc if n > 1 else need)


def _scale_type(format: str):
    if format not in _FORMATS:
        raise ValueError('format must be "int4" or "fp4"')
    return torch.bfloat16 if format == "int4" else _E8M0


def weight_quant(W, *, format: str = "int4", group: int | None = None, zeros: bool = False, values=False,
                 codes=None, scales=None, zeros_out=None, stream=None):
    """Round W [n, k] to 4 bits: returns (codes, scales, zeros, values).

    format="int4": groups of 32, 64 or 128 columns (128 where None), scales in
    bfloat16 [n, groups], and with zeros=True zero points in uint8 [n, groups];
    format="fp4": e2m1 floats in groups of 32, scales in float8_e8m0fnu.  codes
    is uint8 [n, bytes], two codes a byte, its rows padded to 16 bytes.
    values=True (or a tensor): also what the codes stand for, in W's type.
    zeros and values are None where they were not asked for.
    """
    if stream is not None:
        return _on(stream, weight_quant, W, format=format, group=group, zeros=zeros, values=values,
                   codes=codes, scales=scales, zeros_out=zeros_out)
    lib = _lib or _bind()
    ty = _float_type(W, "W")
    whole = 0
    at = _gpu(W)
    n, k, ldw = _rows(W, "W")
    st_type = _scale_type(format)
    if group is None:
        group = 128 if format == "int4" else 32
    if group < 1:
        raise ValueError("group must be positive")
    groups = -(-k // group)
    if codes is None:
        codes = W.new_empty((n, (k + 31) // 32 * 16), dtype=torch.uint8)
        whole = _WHOLE_ROWS                                     # the same bytes on every run, the padding too
    if codes.shape[0] != n:
        raise ValueError(f"codes must have {n} rows")
    ldc = _codes(codes, k)[1]
    if scales is None:
        scales = W.new_empty((n, groups), dtype=st_type)
    lds = _rows(scales, "scales", st_type, (n, groups))[2]
    zp = vp = None
    ldz = ldv = 0
    if zeros:
        if zeros_out is None:
            zeros_out = W.new_empty((n, groups), dtype=torch.uint8)
        ldz = _rows(zeros_out, "zeros_out", torch.uint8, (n, groups))[2]
        zp = zeros_out.data_ptr()
    elif zeros_out is not None:
        raise ValueError("zeros_out needs zeros=True")
    if values is True:
        values = torch.empty_like(W)
    elif values is False:
        values = None
    if values is not None:
        ldv = _rows(values, "values", W.dtype, (n, k))[2]
        vp = values.data_ptr()
    s = _place(at, (codes, scales, zeros_out, values))
    st = lib.batchlas_weight_quant(ty, _FORMATS[format] + whole, group, n, k, W.data_ptr(), ldw, codes.data_ptr(), ldc,
                                   scales.data_ptr(), lds, zp, ldz, vp, ldv, s)
    if st:
        _check(st)
    return codes, scales, zeros_out, values


def weight_matvec(x, codes, scales, zeros=None, *, format: str = "int4", group: int | None = None,
                  x_scales=None, out=None, out_dtype=None, workspace=None, stream=None):
    """y = x W^T for x [m, k] and 4-bit weights as weight_quant gives them.

    x is bfloat16 or float16, or float8_e4m3fn with x_scales as rmsnorm_quant
    gives them (float32 [m], or float8_e8m0fnu [m, ceil(k / 32)]).  y [m, n] is
    `out`, or a new tensor of out_dtype (x's type, bfloat16 for 8-bit x).
    workspace: a uint8 tensor of weight_matvec_workspace(m, k) bytes (0 up to 16
    rows), allocated by the call where it is None.
    """
    if stream is not None:
        return _on(stream, weight_matvec, x, codes, scales, zeros, format=format, group=group,
                   x_scales=x_scales, out=out, out_dtype=out_dtype, workspace=workspace)
    lib = _lib or _bind()
    xt = _TYPES.get(x.dtype, -1)
    if xt < 1:
        raise TypeError(f"x must be bfloat16, float16 or float8_e4m3fn, not {x.dtype}")
    if x.requires_grad or scales.requires_grad or (x_scales is not None and x_scales.requires_grad) \
            or forward_ad._current_level >= 0:
        _refuse_gradients(x, scales, x_scales)
    at = _gpu(x)
    m, k, ldx = _rows(x, "x")
    st_type = _scale_type(format)
    if group is None:
        group = 128 if format == "int4" else 32
    if group < 1:
        raise ValueError("group must be positive")
    groups = -(-k // group)
    n, ldc = _codes(codes, k)
    lds = _rows(scales, "scales", st_type, (n, groups))[2]
    zp = xp = None
    ldz = ldxs = xs = 0
    if zeros is not None:
        ldz = _rows(zeros, "zeros", torch.uint8, (n, groups))[2]
        zp = zeros.data_ptr()
    if xt == 3:
        if x_scales is None:
            raise ValueError("8-bit x needs x_scales")
        if x_scales.dtype is torch.float32:
            xs, xp = 1, _vector(x_scales, "x_scales", torch.float32, m)
        else:
            xs, ldxs = 2, _rows(x_scales, "x_scales", _E8M0, (m, (k + 31) // 32))[2]
            xp = x_scales.data_ptr()
    elif x_scales is not None:
        raise ValueError("x_scales is for 8-bit x")
    if out is None:
        out_dtype = out_dtype or (torch.bfloat16 if xt == 3 else x.dtype)
        out = x.new_empty((*x.shape[:-1], n), dtype=out_dtype)
    yt = _float_type(out, "out")
    ldy = _rows(out, "out", out_dtype, (m, n))[2]
    wp = None
    size = 0
    if workspace is not None:
        size = workspace.numel()
        wp = _vector(workspace, "workspace", torch.uint8, size)
    elif m > 16:
        size = weight_matvec_workspace(m, k)
        workspace = x.new_empty(size, dtype=torch.uint8)
        wp = workspace.data_ptr()
    s = _place(at, (codes, scales, zeros, x_scales, out, workspace))
    st = lib.batchlas_weight_matvec(xt, xs, yt, _FORMATS[format], group, m, n, k, x.data_ptr(), ldx, xp, ldxs,
                                    codes.data_ptr(), ldc, scales.data_ptr(), lds, zp, ldz, out.data_ptr(), ldy, wp, size, s)
    if st:
        _check(st)
    return out


@functools.lru_cache(maxsize=1024)
def weight_matvec_workspace(m: int, k: int) -> int:
    """Bytes of workspace that weight_matvec of this size needs (host-only)."""
    lib = _lib or _bind()
    size = ctypes.c_int64()
    st = lib.batchlas_weight_matvec_workspace(m, k, ctypes.byref(size))
    if st:
        _check(st)
    return size.value
