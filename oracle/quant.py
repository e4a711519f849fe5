"""fp64 oracle of the norms of queries and keys and of the cache in 4 bits.
TEST INFRASTRUCTURE, like the rest of this package: numpy from the definitions,
no code shared with the library.
"""
from __future__ import annotations

import numpy as np

from . import serve

GROUP = 32
LIMITS = {"f16": (2.0 ** -24, 1.25 * 2.0 ** 11), "bf16": (2.0 ** -120, 1.25 * 2.0 ** 123), "f32": (2.0 ** -120, 1.25 * 2.0 ** 123)}


def norm(x, w=None, eps=1e-6, offset=0.0):
    """x [..., hd] / sqrt(mean x^2 + eps) * (w + offset); w None: 1."""
    x = np.asarray(x, np.float64)
    v = 1.0 if w is None else np.asarray(w, np.float64) + offset
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * v


def norm_rotary(x, w, pos, freq, scale=1.0, interleaved=False, eps=1e-6, offset=0.0):
    return serve.rotary(norm(x, w, eps, offset), pos, freq, scale, interleaved)


def norm_rotary_bwd(g, x, w, pos, freq, scale=1.0, interleaved=False, eps=1e-6, offset=0.0):
    """(dx, dw) of norm_rotary by the Jacobian of x / |x|: with n = x r, dn/dx = r (1 - n n^T / hd)."""
    x = np.asarray(x, np.float64)
    g = serve.rotary(g, pos, freq, scale, interleaved, backward=True)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    v = 1.0 if w is None else np.asarray(w, np.float64) + offset
    n, gv = x * r, g * v
    dx = r * (gv - n * np.mean(gv * n, -1, keepdims=True))
    return dx, (g * n).reshape(-1, x.shape[-1]).sum(0)


def quantise(x, dtype):
    """(codes [..., hd] 0..15, scales [..., hd / 32]) of rows x [..., hd] that dtype holds as they are; one group at a
    time."""
    floor, most = LIMITS[dtype]
    rows = np.asarray(x, np.float64).reshape(-1, GROUP)
    codes, scales = np.full(rows.shape, 8, np.int64), np.zeros(len(rows))
    for k, g in enumerate(rows):
        if not np.isfinite(g).all():
            scales[k] = np.nan
            continue
        m = max(g, key=lambda v: (abs(v), v > 0))
        s = m / -8.0
        if s == 0.0:
            continue
        step = max(2.0 ** (np.floor(np.log2(abs(s))) - 4), floor)
        s = np.clip(np.rint(s / step) * step, -most, most)
        scales[k] = s
        if s != 0.0:
            codes[k] = np.clip(np.rint(g / s), -8, 7) + 8
    return codes.reshape(np.shape(x)), scales.reshape(*np.shape(x)[:-1], -1)


def pack(codes):
    """Two codes a byte, an even channel in the low half."""
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).astype(np.uint8)


def unpack(data):
    data = np.asarray(data).astype(np.int64)
    return np.stack((data % 16, data // 16), -1).reshape(*data.shape[:-1], -1)


def values(codes, scales):
    """What codes [..., hd] under scales [..., hd / 32] stand for."""
    return (np.asarray(codes, np.float64) - 8.0) * np.repeat(np.asarray(scales, np.float64), GROUP, -1)
