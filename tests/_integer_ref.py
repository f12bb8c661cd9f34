"""The 8-bit-integer layer operators from their definitions, on the CPU in 64 bits,
and how far a computation in 32 bits may be from them."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24                        # half a step of 32 bits, relative
TINY = np.float32(2.0 ** -126)


def f64(t) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def smallest(dtype) -> float:
    """Half of the smallest subnormal step."""
    info = torch.finfo(dtype)
    return info.tiny * info.eps / 2


# ---------------------------------------------------------------- rounding and products

def quant(x: np.ndarray, given=None):
    """(codes, scales) of float32 x; the quotients in 64 bits, which hold them closely enough for any half."""
    x = x.astype(np.float32)
    if given is None:
        top = np.abs(x).max(1)
        with np.errstate(all="ignore"):
            scale = np.where(np.isfinite(top), np.maximum(top / np.float32(127), TINY), np.float32(np.nan))
        scale = scale.astype(np.float32)
    else:
        scale = given.astype(np.float32)
    good = np.isfinite(scale) & (scale >= TINY)
    with np.errstate(all="ignore"):
        q = np.rint(x.astype(np.float64) / np.where(good, scale, 1).astype(np.float64)[:, None])
    q = np.where(np.isnan(q) | ~good[:, None], 0, np.clip(q, -127, 127))
    return q.astype(np.int8), scale


def product(x: np.ndarray, w: np.ndarray) -> np.ndarray:
    """Sums of int8 products, exact: float64 holds integers up to 2^53."""
    return x.astype(np.float64) @ w.astype(np.float64).T


# ---------------------------------------------------------------- norms around a block
# Statistics in 32 bits: a sum of squares goes through chains of at most 8 products, 8
# vectors, 6 lane exchanges and 8 wavefronts, so it is off by at most 30 u, a mean with eps by
# 32, its inverse root by 16 and the root's own rounding: 17 u.  A product more each for
# the value, the weight, the gate and the sum with the residual: 24 u in all.
K = 24


def spread(gate, rows: int):
    """The gate of every row, or 1."""
    return 1.0 if gate is None else np.repeat(np.atleast_2d(gate), rows // np.atleast_2d(gate).shape[0], 0)


def inverse_rms(v, eps):
    return 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def block_norm(y, x, w, post, gate, c, eps):
    """(h, v, and how far 32 bits may be from each)."""
    g = spread(gate, y.shape[0])
    u = y if post is None else post * y * inverse_rms(y, eps)
    h = c * x + g * u
    r = inverse_rms(h, eps)
    v = w * h * r
    # c is rounded to 32 bits as well: one more
    eh = (K + 1) * U * (np.abs(c * x) + np.abs(g * u))
    # rms(h) moves with h by at most the 2-norm of its error
    move = np.sqrt((eh * eh).mean(1, keepdims=True)) * r
    ev = np.abs(w) * r * eh + np.abs(v) * (1.01 * move + K * U)
    return h, v, eh, ev


def block_norm_grad(dv, y, h, w, post, gate, dh, c, eps):
    """{name: (value, how far 32 bits may be from it)}; the roots as above (17 u), dot products 30 u of the sum
    of magnitudes, and a few products: at most 72 u of the magnitudes that are added."""
    rows, n = h.shape
    kk = 72 * U
    g = spread(gate, rows)
    s = inverse_rms(h, eps)
    unit = h * s
    a = s * (dv * w - unit * (dv * w * unit).mean(1, keepdims=True))
    ea = kk * (s * np.abs(dv * w) + s * np.abs(unit) * np.abs(dv * w * unit).mean(1, keepdims=True))
    if dh is not None:
        a = a + dh
        ea = ea + U * (np.abs(dh) + np.abs(a))
    long = (24 + rows) * U                       # a sum over all rows, in any order
    out = {"dx": (c * a, abs(c) * ea + 2 * U * np.abs(c * a)),
           "dweight": ((dv * unit).sum(0), long * np.abs(dv * unit).sum(0))}
    b = a * g
    if post is None:
        yu, p = y, 1.0
        out["dy"] = (b, np.abs(g) * ea + U * np.abs(b))
    else:
        t = inverse_rms(y, eps)
        yu, p = y * t, post
        mean = (b * p * yu).mean(1, keepdims=True)
        off = (np.abs(g * p * yu) * ea).mean(1, keepdims=True) + kk * np.abs(b * p * yu).mean(1, keepdims=True)
        out["dy"] = (t * (b * p - yu * mean),
                     t * (np.abs(g * p) * ea + kk * np.abs(b * p) + np.abs(yu) * (off + kk * np.abs(mean))))
        out["dpost_weight"] = ((b * yu).sum(0), (np.abs(g * yu) * ea + long * np.abs(b * yu)).sum(0))
    if gate is not None:
        gates = np.atleast_2d(gate).shape[0]
        d = a * p * yu
        e = np.abs(p * yu) * ea + long * np.abs(d)
        fold = lambda t: t.reshape(gates, rows // gates, n).sum(1)  # noqa: E731
        dg, eg = fold(d), fold(e)
        out["dgate"] = (dg[0], eg[0]) if gate.ndim == 1 else (dg, eg)
    return out
