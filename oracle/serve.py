"""fp64 definitions of the serving operators around the retained cache: norm
and rotation of queries and keys, the 4-bit rows, and attention over them.
Plain numpy, one head at a time."""

from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the finite e4m3 values, ascending; index = byte
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119])


def nearest_even(x, grid):
    """Index of the grid value nearest to each x >= 0; a tie goes to the even index."""
    x = np.asarray(x, dtype=np.float64)
    up = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    over, under = grid[up] - x, x - grid[up - 1]
    take = (over < under) | ((over == under) & (up % 2 == 0))
    return np.where(take, up, up - 1)


def quantise(x):
    """x [..., D] fp64 (bf16 values) -> (codes [..., D], scale bytes [..., D/16])."""
    g = np.asarray(x, dtype=np.float64)
    g = np.where(np.isnan(g), 0.0, g)
    g = g.reshape(*g.shape[:-1], g.shape[-1] // 16, 16)
    a = np.abs(g)
    sb = nearest_even(np.minimum(a.max(-1) / 6.0, 448.0), E4M3)
    s = E4M3[sb][..., None]
    # the quotient of an 8-bit and a 4-bit value is a border between codes only where it is exact
    some = s > 0
    mag = nearest_even(np.where(some, np.minimum(a, 6.0 * s), 0.0) / np.where(some, s, 1.0), E2M1)
    code = mag + 8 * np.signbit(g)
    return code.reshape(*code.shape[:-2], 16 * code.shape[-2]).astype(np.uint8), sb.astype(np.uint8)


def values(code, sb):
    v = E2M1[code & 7] * np.where(code >= 8, -1.0, 1.0)
    v = v.reshape(*v.shape[:-1], v.shape[-1] // 16, 16) * E4M3[sb][..., None]
    return v.reshape(*v.shape[:-2], 16 * v.shape[-2])


def held(x):
    """What the 4-bit cache holds for rows x [..., D]."""
    return values(*quantise(x))


def norm_rope(x, weight, eps, inv_freq, pos, R, interleaved):
    """x [T, D] of one head, pos [T] -> [T, D]."""
    y = np.asarray(x, dtype=np.float64).copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    if R:
        ang = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
        # the product is 2^-53 of the angle off; cos and sin of the host take whole turns off exactly
        c, s = np.cos(ang), np.sin(ang)
        i = np.arange(R // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        y[:, a], y[:, b] = y[:, a] * c - y[:, b] * s, y[:, b] * c + y[:, a] * s
    return y


def attention(q, k, v, pos, q_pos):
    """q [T, D], rows k, v [n, D] with positions pos, query positions q_pos [T].
    Returns out [T, D], lse [T], and sum p|v| / sum p (the scale of an error in p)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    T, D = q.shape
    out, mag, lse = np.zeros((T, D)), np.zeros((T, D)), np.full(T, -np.inf)
    for t in range(T):
        see = (pos >= 0) & (pos <= q_pos[t])
        if not see.any():
            continue
        x = k[see] @ q[t] / math.sqrt(D)
        m = x.max()
        p = np.exp(x - m)
        out[t], mag[t] = p @ v[see] / p.sum(), p @ np.abs(v[see]) / p.sum()
        lse[t] = m + math.log(p.sum())
    return out, lse, mag
