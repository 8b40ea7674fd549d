"""Checks of the attentions against the fp64 definition, shared by their tests.

Bounds, per output element, with p the softmax weights of a query:
 - bf16 rounding of the result: 2^-8 |out|;
 - weights rounded for the product with the values: relative `w`, and `floor` times the
   largest weight for each row, numerator only;
 - scores off by dx: weights off by dx relatively, numerator and denominator;
 - the rounding may move by the last two.
dx: fp32 sums of products below 2^-18 A, A the largest sum |q||k| / sqrt(D); a query
rounded to `qr` of its row's largest value, qr * max|q| * sum|k| / sqrt(D); the
hyperbolic tangent 2^-20 (1e-6) of the score; a bias 2^-22 of itself (slope, product
and sum), where the rows count whose weight is not below e^-60 of the largest; the
exponential's argument and result 2^-20.
lse: dx + 2^-20 |lse| + 2^-20.
"""

import math

import numpy as np
import torch

from oracle import serve as O


def f64(t):
    return t.detach().double().cpu().numpy()


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def slopes_of(H, on):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H).float() if on else None


def check(q, k, v, see, far, cap, slope, out, lse, w, floor, qr, what):
    """One head: q [T, D]; k, v [n, D] (what is not seen is ignored); see, far [T, n]."""
    D = q.shape[1]
    some = see.any(0)
    k, v = np.where(some[:, None], k, 0.0), np.where(some[:, None], v, 0.0)
    ref, rl, mag, x = O.attention_of(q, k, v, see, cap, slope, far)
    empty = ~see.any(1)
    assert np.array_equal(empty, np.isneginf(lse)), what
    assert np.all(out[empty] == 0), what
    if empty.all():
        return
    A = float((np.abs(q) @ np.abs(k).T)[see].max(initial=0.0)) / math.sqrt(D)
    Aq = float((np.abs(q).max(1)[:, None] * np.abs(k).sum(1)[None])[see].max(initial=0.0)) / math.sqrt(D)
    dx = A * 2.0 ** -18 + Aq * qr + 2.0 ** -20
    if cap:
        dx += cap * 2.0 ** -20
    if slope:
        top = x.max(1, initial=-np.inf)
        counts = see & (x >= np.where(empty, 0, top)[:, None] - 60)
        dx += abs(slope) * float(np.asarray(far)[counts].max(initial=0.0)) * 2.0 ** -22
    n = see.sum(1)[:, None]
    vmax = np.abs(v).max()
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((w + 2 * dx) * mag + n * floor * vmax) + 1e-30
    err = np.abs(out - ref)
    assert np.all(np.isfinite(out)), what
    assert np.all(err <= tol), (what, float((err / tol).max()), float(err.max()))
    live = ~empty
    le = np.abs(lse[live] - rl[live])
    assert np.all(le <= dx + 2.0 ** -20 * np.abs(rl[live]) + 2.0 ** -20), (what, float(le.max()), dx)
    # and as a whole: no element's rounding is above 2^-8, nor are the weights'
    assert np.linalg.norm(out - ref) <= 2.0 ** -7 * max(np.linalg.norm(ref), 1e-30) + dx * 4 * np.linalg.norm(mag), what
