"""The low-bit layer operators from their definitions, on the CPU: the norm, its
gradient and the products in 64 bits, the roundings to 4 bits in IEEE 32-bit
arithmetic (where the header prescribes it)."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
TINY = np.float32(2.0 ** -126)


def f64(t) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def bf16_round(a: np.ndarray) -> np.ndarray:
    """float32 -> bfloat16 (nearest, ties to even) -> float32."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).float().numpy()


def groups(a: np.ndarray, size: int) -> np.ndarray:
    """[rows, k] -> [rows, groups, size], filled up with zeros."""
    rows, k = a.shape
    pad = -k % size
    return np.pad(a, ((0, 0), (0, pad))).reshape(rows, -1, size)


def least_exponent(top: np.ndarray, most: float) -> np.ndarray:
    """The least e in -127..127 with top <= most 2^e, one step at a time from below."""
    e = np.full(top.shape, -127)
    for c in range(-127, 127):
        e = np.where(top > most * 2.0 ** c, c + 1, e)
    return e


# ---------------------------------------------------------------- norm

def norm(h: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    with np.errstate(all="ignore"):
        return w * h / np.sqrt((h * h).mean(1, keepdims=True) + eps)


def norm_grad(dy, h, w, dh, eps):
    n = h.shape[1]
    s = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    dx = s * (dy * w - h * s * s * (dy * w * h).sum(1, keepdims=True) / n)
    return dx + (0 if dh is None else dh), (dy * h * s).sum(0)


# ---------------------------------------------------------------- 4-bit weights

def quant(W: np.ndarray, fmt: str, group: int, zeros: bool):
    """(codes [n, k], scales, zeros or None, values) of float32 W."""
    W = W.astype(np.float32)
    n, k = W.shape
    b = groups(W, group)
    with np.errstate(all="ignore"):
        top = np.abs(b).max(2)
        finite = np.isfinite(b).all(2)
        if fmt == "fp4":
            e = least_exponent(np.where(finite, top, 0).astype(np.float64), 6.0)
            t = b.astype(np.float64) * 2.0 ** -e[:, :, None].astype(np.float64)
            dist = np.abs(t[..., None] - E2M1[:8] * np.where(np.signbit(t), -1, 1)[..., None])
            near = dist.min(-1, keepdims=True)
            tie = dist == near                       # two candidates: the even code
            code = np.where(tie.sum(-1) == 2, np.argmax(tie & (np.arange(8) % 2 == 0), -1), np.argmax(tie, -1))
            code = code + 8 * np.signbit(t)
            scale = np.where(finite, 2.0 ** e.astype(np.float64), np.nan)
            code = np.where(finite[:, :, None], code, 0)
            val = E2M1[code] * scale[:, :, None]
            z = None
        else:
            if zeros:
                lo, hi = np.minimum(b.min(2), 0), np.maximum(b.max(2), 0)
                span = ((hi - lo).astype(np.float32) / np.float32(15)).astype(np.float32)
                finite = finite & np.isfinite(hi - lo)
            else:
                span = (top / np.float32(7)).astype(np.float32)
            scale = np.where(finite, np.maximum(bf16_round(np.where(finite, span, 1)), TINY), np.float32(np.nan))
            z = np.full(scale.shape, 8.0, np.float32)
            if zeros:
                z = np.where(finite, np.clip(np.rint(-lo / scale), 0, 15), 8).astype(np.float32)
            q = np.rint((b / scale[:, :, None]).astype(np.float32))
            u = np.clip(q + z[:, :, None], 0, 15) if zeros else np.clip(q, -8, 7) + 8
            val = ((u - z[:, :, None]) * scale[:, :, None]).astype(np.float32)
            code = np.where(finite[:, :, None], u, 0).astype(np.int64)
    flat = lambda a: a.reshape(n, -1)[:, :k]  # noqa: E731
    return flat(code), scale, (z if zeros else None), flat(val)


def pack(codes: np.ndarray) -> np.ndarray:
    """[n, k] codes -> bytes, rows padded to 16 bytes with 0xee."""
    n, k = codes.shape
    wide = np.zeros((n, k + k % 2), np.uint8)
    wide[:, :k] = codes
    out = np.full((n, (k + 31) // 32 * 16), 0xEE, np.uint8)
    out[:, :(k + 1) // 2] = wide[:, 0::2] | wide[:, 1::2] << 4
    return out


def unpack(packed: np.ndarray, k: int) -> np.ndarray:
    return np.stack((packed & 15, packed >> 4), 2).reshape(packed.shape[0], -1)[:, :k]


def held(codes, scales, zeros, fmt, group, k) -> np.ndarray:
    """The weights that codes [n, k] stand for, in 64 bits."""
    wide = lambda a: np.repeat(a, group, 1)[:, :k]  # noqa: E731
    with np.errstate(all="ignore"):
        if fmt == "fp4":
            return E2M1[codes] * wide(scales)
        return (codes - (8 if zeros is None else wide(zeros.astype(np.float64)))) * wide(scales)
