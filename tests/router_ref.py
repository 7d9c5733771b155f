"""The gate, the norm and int8 rows in 64 bits, from their definitions (no code shared with the library)."""

from __future__ import annotations

import numpy as np

ULP = 2.0 ** -23  # one unit in the last place of binary32, relative, at most


def gate(z, K, mask=None, normalize=True, scale=1.0, balance=0.0):
    """z float64 [S, E] -> dict(idx, weights, count [E + 1], prob, loss, p, d): d the divisor of the chosen p."""
    S, E = z.shape
    routed = np.ones(S, bool) if mask is None else np.asarray(mask) != 0
    idx = np.full((S, K), -1, np.int64)
    p = np.zeros((S, E))
    for g in range(S):
        order = sorted(range(E), key=lambda e: (0 if np.isnan(z[g, e]) else 1, 0.0 if np.isnan(z[g, e]) else -z[g, e], e))
        able = [e for e in order if not z[g, e] == -np.inf]
        routed[g] &= bool(able)
        if not routed[g]:
            continue
        idx[g, :min(K, len(able))] = able[:K]
        with np.errstate(invalid="ignore"):
            e = np.exp(z[g] - z[g, able[0]])
        p[g] = e / e.sum()
    live = idx >= 0
    pk = np.where(live, np.take_along_axis(p, np.maximum(idx, 0), 1), 0.0)
    d = pk.sum(1) if normalize else np.ones(S)
    d = np.where(routed, d, 1.0)
    count = np.array([(idx == e).sum() for e in range(E)] + [routed.sum()], np.int64)
    n = max(int(count[E]), 1)
    prob = p.sum(0) / n
    loss = balance * E * (count[:E] / (K * n) * prob).sum()
    return dict(idx=idx, weights=scale * pk / d[:, None], count=count, prob=prob, loss=loss, p=p, d=d, routed=routed)


def gate_grad(f, idx, dw, dloss, normalize, scale, balance):
    """The logits' gradient from gate()'s results and any ids [S, K], and a bound of its terms' magnitude."""
    p, count = f["p"], f["count"]
    S, E = p.shape
    K = idx.shape[1]
    live = (idx >= 0) & (idx < E) & f["routed"][:, None]
    at = np.clip(idx, 0, E - 1)
    pk = np.where(live, np.take_along_axis(p, at, 1), 0.0)
    d = (pk.sum(1) if normalize else np.ones(S))[:, None]
    d = np.where(d == 0, 1.0, d)
    dw = np.where(live, dw, 0.0)
    a = scale / d * (dw - ((dw * pk).sum(1, keepdims=True) / d if normalize else 0.0))
    big = np.abs(scale) / d * (np.abs(dw) + ((np.abs(dw) * pk).sum(1, keepdims=True) / d if normalize else 0.0))
    n = max(int(count[E]), 1)
    c = dloss * balance * E * count[:E] / (K * n) / n
    dp, mag = np.tile(c, (S, 1)), np.tile(np.abs(c), (S, 1))
    for k in range(K):
        rows = np.nonzero(live[:, k])[0]
        dp[rows, at[rows, k]] += a[rows, k]
        mag[rows, at[rows, k]] += big[rows, k]
    dz = p * (dp - (p * dp).sum(1, keepdims=True))
    return dz, p * (mag + (p * mag).sum(1, keepdims=True))


def far_logits(z):
    """Largest distance of a finite logit from its row's largest."""
    fine = np.isfinite(z)
    if not fine.any():
        return 0.0
    top = np.where(fine, z, -np.inf).max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        return float(np.where(fine, top - z, 0.0).max())


def gate_rel(z):
    """Relative error of a probability in binary32: the fast exponential is off by 2 + 1.173 |x| units at most (CUDA's
    bound), x itself by half a unit of |x|; its share of a sum of E such values (E / 32 + 5 additions, half a unit each),
    a reciprocal and two products."""
    x = far_logits(z)
    return (2 * (2 + 1.173 * x + x / 2) + (z.shape[1] / 32 + 5) / 2 + 4) * ULP


def rms(h, weight, eps):
    """h, weight float64 -> (y, rstd) of the norm."""
    rstd = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h * rstd * weight, rstd


def rms_grad(dy, h, weight, eps, dsum=None):
    """(dh, dweight, bounds of their terms' magnitude)."""
    _, rstd = rms(h, weight, eps)
    gdy = dy * weight
    mean = (gdy * h).mean(1, keepdims=True)
    dh = rstd * (gdy - h * rstd ** 2 * mean)
    mag = rstd * (np.abs(gdy) + np.abs(h) * rstd ** 2 * np.abs(gdy * h).mean(1, keepdims=True))
    if dsum is not None:
        dh, mag = dh + dsum, mag + np.abs(dsum)
    return dh, (dy * h * rstd).sum(0), mag, np.abs(dy * h * rstd).sum(0)


def int8_rows(x):
    """x float32 [rows, width] -> (codes int8, scales float32), bit for bit: binary32 divisions, ties to even."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        most = np.abs(x).max(1)
        scale = (most / np.float32(127)).astype(np.float32)
        q = np.rint(x / np.where(scale > 0, scale, 1)[:, None])
    bad = ~np.isfinite(most)
    scale[bad] = np.nan
    q[bad | (scale == 0)] = 0
    return np.clip(q, -127, 127).astype(np.int8), scale


def gated_order(n):
    """Source row (gate rows, then up rows) of every packed row of n."""
    m = np.arange(n)
    return m // 32 * 16 + m % 16 + np.where(m % 32 >= 16, n // 2, 0)


def product(wq, ws, xq, xs, gated):
    """(y, what a result may be off by in binary32 before it is rounded) of one expert's rows, float64."""
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T
    v = acc * ws.astype(np.float64) * xs.astype(np.float64)[:, None]
    # The products are whole numbers and their sums exact below 2^24; past that each of the K / 16 additions of the
    # tensor cores rounds, by a unit of at most the sum of the magnitudes. Two products with the scales.
    size = np.abs(xq.astype(np.float64)) @ np.abs(wq.astype(np.float64)).T
    steps = np.where(size < 2 ** 24, 0, xq.shape[1] / 16)
    off = np.abs(ws.astype(np.float64) * xs.astype(np.float64)[:, None]) * size * steps * ULP + np.abs(v) * ULP
    if not gated:
        return v, off
    i = np.arange(v.shape[1] // 2)
    at = i // 16 * 32 + i % 16
    g, u = v[:, at], v[:, at + 16]
    with np.errstate(over="ignore"):
        silu = np.where(g < 0, g * np.exp(-np.abs(g)), g) / (1 + np.exp(-np.abs(g)))
    y = silu * u
    # the exponential's 2 + 1.173 |g| units, a sum, a quotient (2 units) and two products; silu's slope is below 1.1
    return y, np.abs(y) * (2 + 1.173 * np.abs(g) + 6) * ULP + 1.1 * off[:, at] * np.abs(u) + np.abs(silu) * off[:, at + 16]
