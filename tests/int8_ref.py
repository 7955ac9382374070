"""Plain numpy forms of the 8-bit (W8A8) operators, for the tests.

Two forms of the row encoders: `rows32` follows the stated fp32 roundings one by
one (numpy's float32 operations round once, as the operators' definition does),
so its 8-bit values are the exact expected ones; `rows64` is the mathematics in
64 bits, which both are held against with derived tolerances.
"""
from __future__ import annotations

import numpy as np

TINY = np.float32(2.0 ** -100)
U32 = 2.0 ** -24    # half a step of binary32, relative
UBF16 = 2.0 ** -8   # half a step of bfloat16, relative


def factors32(d, s=None, gain=None, divide=True):
    """Column factors: s for weights; 1 / s or gain / s otherwise (binary32, one rounding)."""
    c = np.ones(d, np.float32) if gain is None else gain.astype(np.float32)
    if s is None:
        return c
    s = s.astype(np.float32)
    return (c / s).astype(np.float32) if divide else s


def rows32(h, c):
    """(q, scale, largest) of rows h (float32) with factors c, in the stated fp32 steps."""
    with np.errstate(invalid="ignore", over="ignore"):
        v = (h.astype(np.float32) * c[None, :]).astype(np.float32)
        a = np.abs(v).max(axis=1) if v.size else np.zeros(len(h), np.float32)
        bad = ~np.isfinite(v).all(axis=1)
        some = (a >= TINY) & ~bad
        safe = np.where(some, a, np.float32(1))
        inv = (np.float32(127) / safe).astype(np.float32)
        q = np.rint((v * inv[:, None]).astype(np.float32))
        scale = (safe / np.float32(127)).astype(np.float32)
    q = np.where(some[:, None], q, 0).astype(np.int8)
    scale = np.where(some, scale, np.float32(0))
    return q, np.where(bad, np.float32("nan"), scale).astype(np.float32), a


def rows64(h, s=None, gain=None, divide=True, eps=None):
    """(values over the row's unit, scale) in 64 bits: 127 v / a and a / 127 (times 1 / rms)."""
    h = h.astype(np.float64)
    c = np.ones(h.shape[1]) if gain is None else gain.astype(np.float64)
    if s is not None:
        c = c / s.astype(np.float64) if divide else s.astype(np.float64)
    v = h * c[None, :]
    a = np.abs(v).max(axis=1)
    unit = np.where(a > 0, a / 127, 1.0)
    scale = a / 127
    if eps is not None:
        scale = scale / np.sqrt((h * h).mean(axis=1) + eps)
    return v / unit[:, None], scale


def gemm64(xq, xs, wq, ws):
    # |sum| <= 2^29 < 2^53: the fp64 product of the integers is exact
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T
    return acc * (xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :])
