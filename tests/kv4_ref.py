"""The 4-bit cache's format and the rows' norm and rotation, in numpy and 64
bits, for the tests."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
# Every finite non-negative 8-bit scale by its code (0x7f is NaN).
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])[:127]


def nearest(x, grid):
    """Code of the grid value nearest to x >= 0 (the last when above), halfway
    to the even code."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, x, side="left"), np.searchsorted(mid, x, side="right")
    return np.where(lo == hi, lo, lo + lo % 2)


def quantise(x, g):
    """[..., d] float64 holding bf16 values, g -> codes [..., d] 0..15, scale
    codes [..., d / 16], and which blocks hold a NaN.  The two quotients are
    32-bit ones, correctly rounded: exact wherever x lies on a border and g
    is a power of two, and what decides where g only nearly makes it so (1.9
    in 32 bits is 1.9 - 2.4e-8, and 1.484375 = 5 * 0.15625 * 1.9)."""
    f = np.float32
    b = x.reshape(*x.shape[:-1], -1, 16).astype(f)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        amax = np.abs(b).max(-1)             # NaN if any is
        nan = np.isnan(amax)
        s = nearest(np.where(nan, f(0), amax / (f(6) * f(g))).astype(np.float64), E4M3)
        sg = E4M3[s].astype(f) * f(g)
        y = np.where(sg[..., None] > 0, np.abs(b) / np.where(sg > 0, sg, f(1))[..., None], f(0))
        c = nearest(np.where(np.isnan(y), f(0), y).astype(np.float64), E2M1)
    code = c + 8 * np.signbit(b)
    return code.reshape(x.shape), np.where(nan, 0x7F, s), nan


def pages(pool):
    """uint8 [pages, heads, 9 d] -> codes [pages, heads, 16, d], scale codes [pages, heads, 16, d / 16]."""
    n, h, size = pool.shape
    d = size // 9
    c = pool[..., :8 * d].reshape(n, h, 16, d // 2)
    return np.stack([c & 15, c >> 4], -1).reshape(n, h, 16, d), pool[..., 8 * d:].reshape(n, h, 16, d // 16)


def values(codes, scales, g):
    """What codes and scale codes stand for, float64."""
    x = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    table = np.concatenate([E4M3, [np.nan]])
    s = table[scales & 127] * np.where(scales & 128, -1.0, 1.0)
    return x * np.repeat(s, 16, -1) * g


def turned(x, weight, eps, cos_sin, position, interleaved):
    """Norm and rotation of [tokens, heads, d] float64."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    if cos_sin is not None:
        r = cos_sin.shape[1] // 2
        row = np.full((len(position), 2 * r), np.nan)
        ok = (position >= 0) & (position < len(cos_sin))
        row[ok] = cos_sin[position[ok]]
        c, s = row[:, None, :r], row[:, None, r:]
        ia, ib = (np.arange(0, 2 * r, 2), np.arange(1, 2 * r, 2)) if interleaved else (np.arange(r), np.arange(r, 2 * r))
        a, b, x = x[..., ia], x[..., ib], x.copy()
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def turned32(x, weight, eps, cos_sin, position, interleaved):
    """The same in 32 bits, each operation rounded by itself and the squares
    added neighbours first, as the calls document it: float32, to be rounded
    to bf16."""
    f = np.float32
    x = x.astype(f)
    if weight is not None:
        sq = x * x
        while sq.shape[-1] > 1:
            sq = sq[..., 0::2] + sq[..., 1::2]
        x = x * (f(1) / np.sqrt(sq * f(1 / x.shape[-1]) + f(eps))) * weight.astype(f)
    if cos_sin is not None:
        r = cos_sin.shape[1] // 2
        c, s = cos_sin[position][:, None, :r], cos_sin[position][:, None, r:]
        ia, ib = (np.arange(0, 2 * r, 2), np.arange(1, 2 * r, 2)) if interleaved else (np.arange(r), np.arange(r, 2 * r))
        a, b, x = x[..., ia], x[..., ib], x.copy()
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def bf16(x):
    """float64 -> the nearest bf16 value (ties to even), as float64."""
    u = np.asarray(x, dtype=np.float64).astype(np.float32).view(np.uint32).astype(np.uint64)
    out = (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
    return np.where(np.isnan(x), np.nan, out)
