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


# ------------------------------------------------------------------ 8-bit rows
TOP8 = 1.875 * 2.0 ** 127        # the largest magnitude that is held


def finite8(x):
    x = np.asarray(x, dtype=np.float64)
    return np.clip(np.where(np.isnan(x), 0.0, x), -TOP8, TOP8)


def scale8(top):
    """2^k, k the least integer >= -100 with top <= 448 * 2^k."""
    m, e = np.frexp(np.asarray(top, dtype=np.float64) / 448.0)        # exact where top is 448 * 2^k
    k = np.where(m == 0.5, e - 1, e)
    return np.where(top > 0, 2.0 ** np.maximum(k, -100), 2.0 ** -100)


def round8(x, s):
    """x to the nearest e4m3 multiple of s, ties to even."""
    return np.copysign(E4M3[nearest_even(np.minimum(np.abs(x) / s, 448.0), E4M3)] * s, x)


def held8(x):
    """What the 8-bit cache holds for rows x [n, D] written from a block's first row on, and
    the blocks' scales."""
    x = finite8(x)
    n, D = x.shape
    blocks = np.concatenate((x, np.zeros((-n % 16, D)))).reshape(-1, 16 * D)
    s = scale8(np.abs(blocks).max(-1))
    return round8(blocks, s[:, None]).reshape(-1, D)[:n], s


def append8(held, scales, x):
    """Rows held [n0, D] with their blocks' scales, and new rows x: all rows, and scales."""
    held, x, scales = np.asarray(held, dtype=np.float64), finite8(x), list(scales)
    n0 = len(held)
    first = n0 - n0 % 16
    rows = np.concatenate((held[first:], x))
    out, sc = [held[:first]], scales[:first // 16]
    for i in range(0, len(rows), 16):
        block = rows[i:i + 16]
        new = block[n0 - first:] if i == 0 else block
        s = float(scale8(np.abs(new).max() if new.size else 0.0))
        if i == 0 and n0 % 16:
            s = max(s, scales[first // 16])
        out.append(round8(block, s))
        sc.append(s)
    return np.concatenate(out), np.array(sc)


def attention_of(q, k, v, see, cap=0.0, slope=0.0, far=None):
    """q [T, D], k and v [n, D], see [T, n], far [T, n] distances.  Returns out [T, D], lse [T],
    sum p|v| / sum p, and the scores [T, n] (-inf where not seen)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    x = q @ k.T / math.sqrt(q.shape[1])
    if cap:
        x = cap * np.tanh(x / cap)
    if slope:
        x = x - slope * np.asarray(far, dtype=np.float64)
    x = np.where(see, x, -np.inf)
    some = see.any(-1)
    m = np.where(some, x.max(-1, initial=-np.inf), 0.0)
    p = np.exp(x - m[:, None])
    z = np.where(some, p.sum(-1), 1.0)[:, None]
    lse = np.where(some, m + np.log(z[:, 0]), -np.inf)
    return p @ v / z, lse, p @ np.abs(v) / z, x
