"""MXFP4 in 64 bits, from the format's definition (no code shared with the library)."""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TILE = 128


def pack(x):
    """x float64 [rows, width] -> codes uint8 [rows, width], scale codes uint8 [rows, width / 32]."""
    rows, width = x.shape
    v = np.asarray(x, np.float64).reshape(rows, width // 32, 32)
    most = np.abs(v).max(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(np.isfinite(most) & (most > 0), np.frexp(np.where(np.isfinite(most), most, 1.0))[1] - 1, -400)
    s = np.where(np.isfinite(most), np.maximum(0, e + 125), 255).astype(np.int64)
    bad = s == 255
    a = np.abs(np.where(bad[..., None], 0.0, v)) * np.exp2(np.where(bad, 0, 127 - s).astype(np.float64))[..., None]
    # nearest grid value, ties to the even code
    mid = (GRID[1:] + GRID[:-1]) / 2
    low, high = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
    code = np.where(low == high, low, np.where(low % 2 == 0, low, high))
    sign = np.signbit(v) & ~bad[..., None]
    return (code + 8 * sign).astype(np.uint8).reshape(rows, width), s.astype(np.uint8)


def nibbles(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unnibble(q):
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def tiled(s, fill=0):
    """Scale codes [rows, blocks] -> [ceil(rows / 128), ceil(blocks / 4), 512] uint8; absent ones are `fill`, 0 past the width."""
    rows, blocks = s.shape
    out = np.zeros((-(-rows // TILE), -(-blocks // 4), 512), np.uint8)
    for t in range(out.shape[0]):
        for m in range(TILE):
            row = t * TILE + m
            at = (m % 32) * 16 + m // 32 * 4
            line = s[row] if row < rows else np.full(blocks, fill, np.uint8)
            for c in range(out.shape[1]):
                part = line[4 * c:4 * c + 4]
                out[t, c, at:at + len(part)] = part
    return out


def untiled(sf, rows, width):
    m, b = np.arange(rows)[:, None], np.arange(width // 32)[None, :]
    chunks = -(-width // 128)
    return sf.reshape(-1, chunks, 512)[m // TILE, b // 4, (m % 32) * 16 + m % TILE // 32 * 4 + b % 4]


def values(codes, s):
    """float64 values of codes [rows, width] and scale codes [rows, width / 32] (NaN under 255)."""
    rows, width = codes.shape
    mag = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return (mag.reshape(rows, -1, 32) * scale[..., None]).reshape(rows, width)


def gated_rows(n):
    """Source row (gate rows, then up rows) of every packed row of n."""
    m = np.arange(n)
    return m // 32 * 16 + m % 16 + np.where(m % 32 >= 16, n // 2, 0)


def bf16(x):
    """float64 -> nearest bfloat16 value (ties to even), as float64; through binary32 halves would round twice."""
    x = np.asarray(x, np.float64)
    out = x.copy()
    fine = np.isfinite(x) & (x != 0)
    e = np.maximum(np.frexp(x[fine])[1] - 1, -126)
    unit = np.exp2((e - 7).astype(np.float64))
    out[fine] = np.rint(x[fine] / unit) * unit
    return out
