"""The 4-bit retained cache and attention over it, against the fp64 definition.

The cache's values are compared exactly: scale and code are roundings of exact
quotients.  Attention tolerances, per output element, with p the softmax
weights and A the largest sum |q||k| / sqrt(D) of a query's rows:
 - bf16 rounding of the result: 2^-8 |out|;
 - weights rounded to fp16: 2^-11 sum p|v| / sum p; weights too small for fp16's
   normal numbers: half a step, 2^-25, where the largest weight is at least 2^4;
 - scores: fp32 accumulation and the fp16 query (2^-24 of its largest value off):
   below 2^-19 A, and the base-2 exponential's argument and result below 2^-20 of
   it, so weights move by 2^-18 A in relative terms, numerator and denominator;
 - the rounding may move by the last two.
lse: 2^-18 A + 2^-20 |lse| + 2^-20.
"""

import math

import numpy as np
import pytest
import torch

from oracle import kvc_oracle
from oracle import serve as O
from synth import get_config, make_layer_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_score_kv_gb300 import build
    build.build()
    import attention_score_kv_gb300.kvc as kvc
    return kvc


def f64(t):
    return t.detach().double().cpu().numpy()


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def all_rows(K, cache, B, H, D, so):
    """Every row of every slot, [B, rows, D] each."""
    n = [so[h + 1] - so[h] for h in range(H)]
    k, v = (torch.empty((B * so[H], D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K.kvc_read_q4(cache, B, H, D, so, None, n, k, v, out_off=list(so))
    return f64(k).reshape(B, so[H], D), f64(v).reshape(B, so[H], D)


def filled(K, B, H, D, so, n, seed, S=None, scale=1.0):
    """A cache whose heads hold n[h] rows each (positions 0, 3, 6, ...), every other
    byte 0xff (NaN scales); (cache, pos, K rows, V rows as held)."""
    S = S or max(max(n), 1) * 3
    k, v = rnd(seed, B, H, S, D, scale=scale), rnd(seed + 1, B, H, S, D)
    cache, pos = K.q4_cache(B, D, so)
    cache.fill_(0xff)
    idx = torch.full_like(pos, -1).view(B, -1)
    for h in range(H):
        idx[:, so[h]:so[h] + n[h]] = torch.arange(n[h], device="cuda", dtype=torch.int32) * 3 % S
    K.kvc_gather_q4(k, v, idx, B, H, S, D, n, so, cache, pos)
    return cache, pos, k, v


def attend(K, q, cache, pos, rows, extra, q_pos, B, T, Hq, H, D, so, lse=True):
    ws = K.attention_q4_workspace(B, T, Hq, H, D)
    ws.fill_(0xff)
    out = torch.full((B, Hq, T, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full((B, Hq, T), float("nan"), device="cuda") if lse else None
    K.kvc_attention_q4(q, cache, pos, rows, extra, q_pos, B, T, Hq, H, D, so, out, ls, ws)
    return out, ls


def check_attention(K, q, cache, pos, rows, extra, q_pos, B, T, Hq, H, D, so, out, lse, heads=None, batches=None):
    kk, vv = all_rows(K, cache, B, H, D, so)
    q, out, lse = f64(q), f64(out), f64(lse)
    pos, rows, q_pos = (t.cpu().numpy() for t in (pos.view(B, -1), rows.view(B, H), q_pos.view(B, T)))
    G = Hq // H
    for b in batches if batches is not None else range(B):
        for hq in heads if heads is not None else range(Hq):
            h = hq // G
            n = min(max(int(rows[b, h]) + extra, 0), so[h + 1] - so[h])
            k, v, p = kk[b, so[h]:so[h] + n], vv[b, so[h]:so[h] + n], pos[b, so[h]:so[h] + n]
            seen = (p >= 0) & (p <= q_pos[b].max())
            k, v = np.where(seen[:, None], k, 0), np.where(seen[:, None], v, 0)
            ref, rl, mag = O.attention(q[b, hq], k, v, p, q_pos[b])
            A = 0.0 if not seen.any() else float((np.abs(q[b, hq]) @ np.abs(k[seen]).T).max()) / math.sqrt(D)
            vmax = np.abs(v[seen]).max() if seen.any() else 0.0
            tol = 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -11 + A * 2.0 ** -18) * mag + n * 2.0 ** -29 * vmax
            err = np.abs(out[b, hq] - ref)
            assert np.all(err <= tol), (b, hq, float(err.max()), float((err - tol).max()))
            empty = np.isneginf(rl)
            assert np.array_equal(empty, np.isneginf(lse[b, hq]))
            le = np.abs(lse[b, hq][~empty] - rl[~empty])
            assert np.all(le <= 2.0 ** -18 * A + 2.0 ** -20 * np.abs(rl[~empty]) + 2.0 ** -20), (b, hq, le.max())


# ------------------------------------------------------------------ the rows
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_every_kind(K, D):
    """Every bf16 exponent, borders between codes, zeros, subnormals, huge values."""
    B, H, S = 1, 1, 512
    x = rnd(5, S, D).float()
    x[:64] *= torch.exp2(torch.arange(-40, 24, device="cuda"))[:, None]
    border = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6], device="cuda").repeat(D // 8)
    for i in range(64):                     # scales of every mantissa, subnormal ones too
        x[64 + i] = border * (8 + i % 8) * 2.0 ** (i // 8 * 2 - 13)
        x[128 + i] = -x[64 + i]
    x[200] = 0
    x[201, ::16] = 6 * 2.0 ** -10           # half the smallest scale: becomes zeros
    x[202, ::16] = 6 * 2.0 ** -10 * 1.01
    x[203] = 1e-40
    x[204, 0] = 3e38
    x = x.to(torch.bfloat16).view(B, H, S, D)
    y = x.flip(2).contiguous()
    so = K.kvc_q4_layout(H, S, [S], 0)
    cache, pos = K.q4_cache(B, D, so)
    K.kvc_gather_q4(x, y, torch.arange(S, dtype=torch.int32, device="cuda"), B, H, S, D, [S], so, cache, pos)
    k, v = all_rows(K, cache, B, H, D, so)
    K.kvc_check_status()
    assert np.array_equal(k[0], O.held(f64(x)[0, 0])) and np.array_equal(v[0], O.held(f64(y)[0, 0]))
    assert torch.equal(pos, torch.arange(S, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_not_finite(K, D):
    x = rnd(6, 1, 1, 16, D)
    x[0, 0, 1, 3], x[0, 0, 2, 17], x[0, 0, 3, 60] = float("nan"), float("inf"), float("-inf")
    so = [0, 16]
    cache, pos = K.q4_cache(1, D, so)
    K.kvc_gather_q4(x, x, torch.arange(16, dtype=torch.int32, device="cuda"), 1, 1, 16, D, [16], so, cache, pos)
    with pytest.raises(K.KvcError) as ei:
        K.kvc_check_status()
    assert ei.value.code == K.KVC_ERR_DEVICE
    K.kvc_check_status()                    # read once, then clear
    k, v = all_rows(K, cache, 1, 1, D, so)
    want = O.held(f64(x)[0, 0])
    assert k[0, 1, 3] == 0 and k[0, 2, 17] == 2688 and k[0, 3, 60] == -2688
    assert np.array_equal(k[0], want) and np.array_equal(v[0], want)


@pytest.mark.parametrize("B,H,S,D,K_l,extra", [
    (1, 1, 1, 128, [1], 0), (2, 3, 40, 64, [0, 17, 400], 5), (3, 2, 300, 128, [299, 16], 33),
    (2, 5, 77, 128, [1, 15, 16, 31, 33], 0),
])
def test_gather(K, B, H, S, D, K_l, extra):
    so = K.kvc_q4_layout(H, S, K_l, extra)
    kept = [min(n, S) for n in K_l]
    k, v = rnd(1, B, H, S, D, scale=3), rnd(2, B, H, S, D)
    g = torch.Generator().manual_seed(3)
    idx = torch.full((B, so[H]), -7, dtype=torch.int32)
    for b in range(B):
        for h in range(H):
            idx[b, so[h]:so[h] + kept[h]] = torch.sort(torch.randperm(S, generator=g)[:kept[h]]).values.int()
    cache, pos = K.q4_cache(B, D, so)
    cache.fill_(0x5a)
    before = cache.clone().view(B, -1, 18 * D)
    pos.fill_(-9)
    K.kvc_gather_q4(k, v, idx.cuda(), B, H, S, D, K_l, so, cache, pos)
    kk, vv = all_rows(K, cache, B, H, D, so)
    K.kvc_check_status()
    after, pc = cache.view(B, -1, 18 * D), pos.view(B, -1).cpu()
    for b in range(B):
        for h in range(H):
            at, n = idx[b, so[h]:so[h] + kept[h]].long().numpy(), kept[h]
            assert np.array_equal(kk[b, so[h]:so[h] + n], O.held(f64(k)[b, h, at]))
            assert np.array_equal(vv[b, so[h]:so[h] + n], O.held(f64(v)[b, h, at]))
            full = -(-n // 16) * 16          # the last block's rest is zeros, blocks behind it are as they were
            assert not kk[b, so[h] + n:so[h] + full].any() and not vv[b, so[h] + n:so[h] + full].any()
            lo, hi = (so[h] + full) // 16, so[h + 1] // 16
            assert torch.equal(after[b, lo:hi], before[b, lo:hi])
            assert torch.equal(pc[b, so[h]:so[h] + n], idx[b, so[h]:so[h] + n])
            assert torch.all(pc[b, so[h] + n:so[h + 1]] == -9)


@pytest.mark.parametrize("D", [64, 128])
def test_tensors_that_start_on_16_bytes(K, D):
    """Gather, append and read on tensors that start on an odd multiple of 16 bytes."""
    def shifted(t):
        x = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[8:].view(t.shape)
        assert x.data_ptr() % 32 == 16
        return x.copy_(t)

    B, H, S, n, T = 2, 2, 90, [70, 33], 3
    so = K.kvc_q4_layout(H, S, n, 20)
    k, v = rnd(1, B, H, S, D, scale=2), rnd(2, B, H, S, D)
    kt, vt, pt = rnd(3, B, H, T, D), rnd(4, B, H, T, D), i32([[500, 501, 502]] * B)
    idx = torch.arange(so[H], device="cuda", dtype=torch.int32).repeat(B) % S
    rows = i32([n] * B)
    got = []
    for f in (lambda t: t, shifted):
        cache, pos = K.q4_cache(B, D, so)
        cache.zero_()
        K.kvc_gather_q4(f(k), f(v), idx, B, H, S, D, n, so, cache, pos)
        K.kvc_append_q4(f(kt), f(vt), pt, B, H, T, D, so, rows, cache, pos)
        ko, vo = (f(torch.zeros((B * (sum(n) + 2 * T), D), dtype=torch.bfloat16, device="cuda")) for _ in range(2))
        K.kvc_read_q4(cache, B, H, D, so, None, [x + T for x in n], ko, vo)
        got.append((cache, pos, ko, vo))
    K.kvc_check_status()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert np.array_equal(f64(got[0][2][n[0]:n[0] + T]), O.held(f64(kt)[0, 0]))


def test_gather_records_a_position_outside(K):
    k = rnd(1, 1, 1, 20, 64)
    for bad in (-1, 20, 2 ** 31 - 1):
        cache, pos = K.q4_cache(1, 64, [0, 16])
        idx = i32([0, 1, bad] + [0] * 13)
        K.kvc_gather_q4(k, k, idx, 1, 1, 20, 64, [3], [0, 16], cache, pos)
        with pytest.raises(K.KvcError) as ei:
            K.kvc_check_status()
        assert ei.value.code == K.KVC_ERR_DEVICE


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,first", [(1, 0), (1, 1), (1, 15), (1, 16), (2, 7), (3, 14), (5, 31), (16, 8), (17, 0),
                                     (33, 15), (40, 1)])
def test_append_writes_its_rows_and_no_other(K, D, T, first):
    B, H = 2, 3
    so = [0, 80, 80 + 96, 80 + 96 + 80]
    cache, pos, _, _ = filled(K, B, H, D, so, [80, 96, 80], 9)
    K0, V0 = all_rows(K, cache, B, H, D, so)
    p0 = pos.clone().view(B, -1).cpu().numpy()
    rows = np.array([[first, first + 1, first + 2], [first + 3, first + 5, first + 8]])
    k, v = rnd(11, B, H, T, D, scale=4), rnd(12, B, H, T, D)
    pn = np.arange(B * T).reshape(B, T) + 1000
    pn[1, T // 2] = -5                       # an absent token
    K.kvc_append_q4(k, v, i32(pn), B, H, T, D, so, i32(rows), cache, pos)
    K1, V1 = all_rows(K, cache, B, H, D, so)
    K.kvc_check_status()
    want_k, want_v, want_p = K0.copy(), V0.copy(), p0.copy()
    for b in range(B):
        for h in range(H):
            for t in range(T):
                r = so[h] + rows[b, h] + t
                gone = pn[b, t] < 0
                want_k[b, r] = 0 if gone else O.held(f64(k)[b, h, t])
                want_v[b, r] = 0 if gone else O.held(f64(v)[b, h, t])
                want_p[b, r] = -1 if gone else pn[b, t]
    assert np.array_equal(K1, want_k) and np.array_equal(V1, want_v)
    assert np.array_equal(pos.view(B, -1).cpu().numpy(), want_p)


def test_append_without_room_leaves_the_head(K):
    B, H, D, so = 2, 2, 128, [0, 32, 64]
    cache, pos, _, _ = filled(K, B, H, D, so, [32, 32], 3)
    k = rnd(1, B, H, 3, D)
    before, pb = all_rows(K, cache, B, H, D, so), pos.clone()
    for rows in ([[30, 30], [32, -1]], [[2 ** 31 - 1, -2 ** 31], [31, 99]]):
        K.kvc_append_q4(k, k, i32([[1, 2, 3]] * 2), B, H, 3, D, so, i32(rows), cache, pos)
        with pytest.raises(K.KvcError) as ei:
            K.kvc_check_status()
        assert ei.value.code == K.KVC_ERR_DEVICE
        after = all_rows(K, cache, B, H, D, so)
        assert np.array_equal(before[0], after[0]) and np.array_equal(before[1], after[1]) and torch.equal(pb, pos)
    K.kvc_append_q4(k, k, i32([[1, 2, 3]] * 2), B, H, 3, D, so, i32([[29, 30], [0, 0]]), cache, pos)   # one head full
    with pytest.raises(K.KvcError):
        K.kvc_check_status()
    after = all_rows(K, cache, B, H, D, so)
    assert np.array_equal(after[0][0, 29:32], O.held(f64(k)[0, 0]))
    assert np.array_equal(after[0][0, 32:], before[0][0, 32:])


@pytest.mark.parametrize("D", [64, 128])
def test_read_ranges(K, D):
    B, H, so = 2, 2, [0, 48, 128]
    cache, pos, k, v = filled(K, B, H, D, so, [48, 80], 21)
    kk, vv = all_rows(K, cache, B, H, D, so)
    n, first, oo = [5, 33], np.array([[0, 13], [43, 47]]), [2, 10, 50]
    ko = torch.full((B * oo[2], D), 77.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    K.kvc_read_q4(cache, B, H, D, so, i32(first), n, ko, vo, out_off=oo)
    K.kvc_check_status()
    want_k, want_v = np.full((B, oo[2], D), 77.0), np.full((B, oo[2], D), 77.0)
    for b in range(B):
        for h in range(H):
            r = so[h] + first[b, h]
            want_k[b, oo[h]:oo[h] + n[h]], want_v[b, oo[h]:oo[h] + n[h]] = kk[b, r:r + n[h]], vv[b, r:r + n[h]]
    assert np.array_equal(f64(ko).reshape(want_k.shape), want_k)
    assert np.array_equal(f64(vo).reshape(want_v.shape), want_v)


def test_read_outside_a_slot_gives_zeros(K):
    D, so = 128, [0, 32, 64]
    cache, _, _, _ = filled(K, 1, 2, D, so, [32, 32], 22)
    kk, _ = all_rows(K, cache, 1, 2, D, so)
    for first, want in ([[-3, 30]], None), ([[2 ** 31 - 2, -2 ** 31]], 0):
        ko, vo = (torch.full((12, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        K.kvc_read_q4(cache, 1, 2, D, so, i32(first), [6, 6], ko, vo)
        with pytest.raises(K.KvcError):
            K.kvc_check_status()
        if want is None:
            got = f64(ko)
            assert not got[:3].any() and np.array_equal(got[3:6], kk[0, :3])
            assert np.array_equal(got[6:8], kk[0, 62:64]) and not got[8:].any()
        else:
            assert not f64(ko).any() and not f64(vo).any()


# ------------------------------------------------------------------ attention
ATT = [
    # B, T, Hq, H, D, rows per head
    (1, 1, 1, 1, 128, [1]),
    (1, 1, 4, 1, 64, [16]),
    (2, 1, 8, 2, 128, [17, 300]),
    (3, 1, 10, 2, 64, [0, 129]),            # a head that holds nothing
    (1, 1, 32, 8, 128, [1000, 15, 16, 33, 2500, 1, 700, 64]),
    (2, 2, 14, 2, 128, [47, 205]),          # 14 query rows
    (1, 3, 12, 3, 64, [31, 32, 600]),
    (2, 5, 8, 2, 128, [100, 260]),          # 20
    (1, 16, 5, 1, 128, [333]),              # 80
    (1, 40, 4, 2, 64, [90, 41]),
    (1, 130, 6, 2, 128, [140, 1000]),
    (1, 300, 3, 1, 64, [777]),
    (70, 1, 4, 2, 128, [40, 90]),
    # more heads than clusters hold, heads without rows among them, and a slot too long for a cluster
    (41, 2, 8, 2, 64, [0, 129]),
    (40, 1, 5, 1, 128, [3]),
    (20, 1, 14, 2, 128, [17, 700]),
    (1, 1, 8, 2, 128, [17000, 5]),
    (1, 2, 6, 2, 64, [33, 20000]),
]


@pytest.mark.parametrize("case", ATT)
@pytest.mark.parametrize("sharp", [0.5, 8.0])
def test_attention(K, case, sharp):
    B, T, Hq, H, D, n = case
    so = K.kvc_q4_layout(H, 1 << 20, n, T + 20)
    cache, pos, _, _ = filled(K, B, H, D, so, n, 31, scale=1.5)
    rows = np.array(n)[None, :] - np.minimum(np.arange(B)[:, None] % 5, np.array(n))     # ragged batch
    top = 3 * max(max(n), 1)
    new = top + np.arange(T)[None, :] + 10 * np.arange(B)[:, None]
    # the new tokens join the cache, so that queries see them causally
    k, v = rnd(41, B, H, T, D, scale=1.5), rnd(42, B, H, T, D)
    K.kvc_append_q4(k, v, i32(new), B, H, T, D, so, i32(rows), cache, pos)
    q = rnd(43, B, Hq, T, D, scale=sharp)
    args = (q, cache, pos, i32(rows), T, i32(new), B, T, Hq, H, D, so)
    out, lse = attend(K, *args)
    K.kvc_check_status()
    check_attention(K, *args, out, lse)
    again, lse2 = attend(K, *args)                       # the same bits
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    bare, _ = attend(K, *args, lse=False)
    assert torch.equal(out, bare)


# Many query rows, with one CTA per tile of them (more tiles than SMs) and with several; every CTA
# goes through many tiles of cache rows, and new tokens end in the middle of one.
LONG = [
    (20, 66, 8, 8, 64, [700, 130, 1000, 128, 1, 511, 640, 333]),
    (24, 70, 14, 7, 128, [900, 700, 1200, 65, 1290, 128, 256]),
    (1, 300, 8, 8, 128, [3000, 2950, 100, 0, 2047, 2048, 2049, 1500]),
    (2, 130, 6, 2, 64, [9000, 7001]),
]


@pytest.mark.parametrize("case", LONG)
@pytest.mark.parametrize("sharp", [0.5, 8.0])
def test_attention_of_many_rows_over_many_tiles(K, case, sharp):
    B, T, Hq, H, D, n = case
    so = K.kvc_q4_layout(H, 1 << 20, n, T + 20)
    cache, pos, _, _ = filled(K, B, H, D, so, n, 131, scale=1.5)
    rows = np.array(n)[None, :] - np.minimum(np.arange(B)[:, None] % 5, np.array(n))
    new = 3 * max(n) + np.arange(T)[None, :] + 10 * np.arange(B)[:, None]
    k, v = rnd(141, B, H, T, D, scale=1.5), rnd(142, B, H, T, D)
    K.kvc_append_q4(k, v, i32(new), B, H, T, D, so, i32(rows), cache, pos)
    holes = torch.rand(pos.shape, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda") < 0.01
    pos[holes] = -1                                      # masked rows in every tile
    q = rnd(143, B, Hq, T, D, scale=sharp)
    args = (q, cache, pos, i32(rows), T, i32(new), B, T, Hq, H, D, so)
    out, lse = attend(K, *args)
    K.kvc_check_status()
    check_attention(K, *args, out, lse, batches=sorted({0, B - 1}))
    again, lse2 = attend(K, *args)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("T", [1, 6, 70])
@pytest.mark.parametrize("D", [64, 128])
def test_masks_that_leave_rows_empty(K, T, D):
    """Queries before every position, rows with negative positions, heads without rows,
    and bytes of unseen rows that decode to NaN."""
    B, H, Hq, n = 2, 2, 6, [100, 37]
    so = K.kvc_q4_layout(H, 1000, n, 30)
    cache, pos, _, _ = filled(K, B, H, D, so, n, 51)
    pv = pos.view(B, -1)
    pv[0, so[0]:so[0] + 50] = -1                         # holes
    pv[1, so[1]:so[1] + 37] = -4                         # nothing left of a head
    pv[0, so[1]:so[1] + 37:2] = 2 ** 31 - 1              # seen by the last position alone
    rec = cache.view(B, -1, 18 * D)
    rec[0, so[0] // 16:so[0] // 16 + 3] = 0xff           # holes hold NaN scales
    rec[1, so[1] // 16:so[1] // 16 + 2] = 0xff
    rows = i32([n, n])
    qp = np.full((B, T), 150)
    qp[:, ::3] = -1                                      # sees nothing
    qp[0, T // 2] = 2 ** 31 - 1
    q = rnd(53, B, Hq, T, D)
    args = (q, cache, pos, rows, 0, i32(qp), B, T, Hq, H, D, so)
    out, lse = attend(K, *args)
    K.kvc_check_status()
    check_attention(K, *args, out, lse)
    assert torch.all(out[1, 3:] == 0) and torch.isneginf(lse[1, 3:]).all()
    none = attend(K, q, cache, pos, i32(np.zeros((B, H))), 0, i32(qp), B, T, Hq, H, D, so)
    assert torch.all(none[0] == 0) and torch.isneginf(none[1]).all()


def test_positions_in_any_order(K):
    """Rows behind later ones may have earlier positions; every query row has a mask of its own."""
    B, T, H, Hq, D, n = 1, 9, 1, 3, 128, [200]
    so = K.kvc_q4_layout(H, 1000, n, 0)
    cache, pos, _, _ = filled(K, B, H, D, so, n, 61)
    pos[:200] = torch.randperm(200, generator=torch.Generator().manual_seed(1)).int().cuda()
    qp = i32([[199, 0, 100, 50, -1, 3, 198, 20, 7]])
    q = rnd(62, B, Hq, T, D, scale=2)
    args = (q, cache, pos, i32([[200]]), 0, qp, B, T, Hq, H, D, so)
    check_attention(K, *args, *attend(K, *args))


def test_a_query_that_is_not_finite_or_extreme(K):
    """NaN and infinity stay in their own query row; zeros, tiny and huge rows are right."""
    B, T, H, Hq, D, n = 1, 1, 1, 7, 128, [90]
    so = K.kvc_q4_layout(H, 1000, n, 0)
    cache, pos, _, _ = filled(K, B, H, D, so, n, 71)
    q = rnd(72, B, Hq, T, D)
    q[0, 1, 0, 3], q[0, 2, 0, 9] = float("nan"), float("inf")
    q[0, 3] = 0
    q[0, 4] *= 1e-30
    q[0, 5] *= 2.0 ** 20
    args = (q, cache, pos, i32([[90]]), 0, i32([[1000]]), B, T, Hq, H, D, so)
    out, lse = attend(K, *args)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1]).all()
    assert torch.isnan(out[0, 2]).any()
    check_attention(K, *args, out, lse, heads=[0, 3, 4, 6])
    # one key takes it all: the row of the largest score
    kk, vv = all_rows(K, cache, B, H, D, so)
    best = (kk[0, :90] @ f64(q)[0, 5, 0]).argmax()
    assert np.all(np.abs(f64(out)[0, 5, 0] - vv[0, best]) <= 2.0 ** -8 * np.abs(vv[0, best]))


def test_counts_outside_the_slot_are_clamped_and_recorded(K):
    B, T, H, Hq, D, so = 1, 1, 2, 4, 64, [0, 32, 64]
    cache, pos, _, _ = filled(K, B, H, D, so, [32, 32], 81)
    q, qp = rnd(82, B, Hq, T, D), i32([[1000]])
    for rows, extra in ([[40, 5]], 0), ([[-3, 5]], 0), ([[30, 30]], 9), ([[2 ** 31 - 1, 8]], 2 ** 31 - 1):
        args = (q, cache, pos, i32(rows), extra, qp, B, T, Hq, H, D, so)
        out, lse = attend(K, *args)
        with pytest.raises(K.KvcError) as ei:
            K.kvc_check_status()
        assert ei.value.code == K.KVC_ERR_DEVICE
        check_attention(K, *args, out, lse)
    # the same for many heads, and for many query rows
    for B, T in (40, 1), (1, 9):
        cache, pos, _, _ = filled(K, B, H, D, so, [32, 32], 83)
        q, qp = rnd(84, B, Hq, T, D), i32(np.full((B, T), 1000))
        for rows, extra in ([[40, 5]], 0), ([[-3, 5]], 1), ([[2 ** 31 - 1, 8]], 2 ** 31 - 1):
            args = (q, cache, pos, i32(rows * B), extra, qp, B, T, Hq, H, D, so)
            out, lse = attend(K, *args)
            with pytest.raises(K.KvcError) as ei:
                K.kvc_check_status()
            assert ei.value.code == K.KVC_ERR_DEVICE
            check_attention(K, *args, out, lse, batches=[0, B - 1])


@pytest.mark.parametrize("B,Hq,H,T", [(300, 4, 4, 1), (1, 8, 1, 1), (5, 6, 3, 4)])
def test_many_heads_and_long_rows(K, B, Hq, H, T):
    """More heads than ranges, one head across all ranges, ranges that end inside heads."""
    D = 64
    n = [6000] if H == 1 else [20 + 60 * h for h in range(H)]
    so = K.kvc_q4_layout(H, 1 << 20, n, 0)
    cache, pos, _, _ = filled(K, B, H, D, so, n, 91)
    rows = i32(np.array(n)[None] - np.arange(B)[:, None] % 20)
    q, qp = rnd(92, B, Hq, T, D, scale=2), i32(np.full((B, T), 1 << 20))
    args = (q, cache, pos, rows, 0, qp, B, T, Hq, H, D, so)
    check_attention(K, *args, *attend(K, *args))


def test_a_wait_that_gives_up_is_reported(K):
    """With a limit of one poll the many-row kernel's waits may give up: the call ends all the
    same, a wait that did give up is reported, and the next call is right."""
    B, T, H, Hq, D, n = 4, 40, 8, 32, 128, [6000] * 8
    so = K.kvc_q4_layout(H, 1 << 20, n, 0)
    cache, pos, _, _ = filled(K, B, H, D, so, n, 96)
    q, qp = rnd(97, B, Hq, T, D), i32(np.full((B, T), 1 << 20))
    args = (q, cache, pos, i32([n] * B), 0, qp, B, T, Hq, H, D, so)
    for limit in (1, 1, 1, 0):
        K.kvc_set_option(K.KVC_OPT_WAIT_LIMIT, limit)
        try:
            out, lse = attend(K, *args)
            gave_up = False
            try:
                K.kvc_check_status()
            except K.KvcError as e:
                assert e.code == K.KVC_ERR_TIMEOUT
                gave_up = True
        finally:
            K.kvc_set_option(K.KVC_OPT_WAIT_LIMIT, 0)
        assert limit or not gave_up
        if not gave_up:
            check_attention(K, *args, out, lse, heads=[0, 31], batches=[0, 3])


def test_offsets_past_32_bits(K):
    """A slot of 2^25 rows, 4.8 GB: append and attention at its far end."""
    D, cap = 128, 1 << 25
    so = [0, cap]
    cache = torch.zeros(cap * D * 9 // 8, dtype=torch.uint8, device="cuda")
    pos = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    k, v, q = rnd(1, 1, 1, 40, D), rnd(2, 1, 1, 40, D), rnd(3, 1, 4, 1, D)
    rows = i32([[cap - 43]])
    K.kvc_append_q4(k, v, i32([np.arange(40)]), 1, 1, 40, D, so, rows, cache, pos)
    ko, vo = (torch.empty((40, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K.kvc_read_q4(cache, 1, 1, D, so, rows, [40], ko, vo)
    out, lse = attend(K, q, cache, pos, rows, 43, i32([[30]]), 1, 1, 4, 1, D, so)
    K.kvc_check_status()
    hk, hv = O.held(f64(k)[0, 0]), O.held(f64(v)[0, 0])
    assert np.array_equal(f64(ko), hk) and np.array_equal(f64(vo), hv)
    for h in range(4):
        ref, rl, mag = O.attention(f64(q)[0, h], hk, hv, np.arange(40), np.array([30]))
        assert np.all(np.abs(f64(out)[0, h] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * mag)
        assert abs(float(lse[0, h, 0]) - rl[0]) < 1e-3


@pytest.mark.parametrize("form,B,T,n", [("cluster", 1, 1, 90), ("ranges", 40, 1, 90), ("many rows", 1, 3, 90),
                                        ("many rows, split", 2, 50, 3000)])
def test_odd_queries_leave_their_neighbours_alone(K, form, B, T, n):
    """Query rows that are not finite, zero, tiny or huge beside ordinary ones, in every form of the
    kernel: NaN and infinity stay in their rows, and every other row is right."""
    H, Hq, D = 1, 7, 128
    so = K.kvc_q4_layout(H, 1 << 20, [n], 0)
    cache, pos, _, _ = filled(K, B, H, D, so, [n], 171)
    rows, qp = i32([[n]] * B), i32(np.full((B, T), 1 << 20))
    plain = rnd(172, B, Hq, T, D)
    plain[:, 3, ::5] = 0
    plain[:, 4, ::5] *= 1e-30
    odd = plain.clone()
    odd[:, 1, ::5, 3], odd[:, 2, ::5, 9] = float("nan"), float("inf")
    odd[:, 5, ::5] *= 2.0 ** 20
    args = (cache, pos, rows, 0, qp, B, T, Hq, H, D, so)
    out, lse = attend(K, odd, *args)
    ref, ref_lse = attend(K, plain, *args)
    K.kvc_check_status()
    assert torch.isnan(out[:, 1, ::5]).all() and torch.isnan(lse[:, 1, ::5]).all()
    assert torch.isnan(out[:, 2, ::5]).any(-1).all()
    # a huge query: one key takes it all, that of the largest score
    kk, vv = all_rows(K, cache, B, H, D, so)
    for b in range(B):
        for t in range(0, T, 5):
            best = vv[b, (kk[b, :n] @ f64(odd)[b, 5, t]).argmax()]
            assert np.all(np.abs(f64(out)[b, 5, t] - best) <= 2.0 ** -8 * np.abs(best))
    same = (plain == odd).all(-1)                        # the rows that are alike in both calls
    assert not same[:, 1, ::5].any() and same[:, 0].all()
    check_attention(K, plain, *args, torch.where(same[..., None], out, ref), torch.where(same, lse, ref_lse),
                    batches=sorted({0, B - 1}))


def test_a_wait_that_gives_up_is_recorded(K):
    """With a limit of one poll some wait gives up (measured: in 56 of 100 calls), and is reported."""
    B, T, H, Hq, D, n = 4, 40, 8, 32, 128, [6000] * 8
    so = K.kvc_q4_layout(H, 1 << 20, n, 0)
    cache, pos, _, _ = filled(K, B, H, D, so, n, 196)
    q, qp = rnd(197, B, Hq, T, D), i32(np.full((B, T), 1 << 20))
    gave_up = False
    K.kvc_set_option(K.KVC_OPT_WAIT_LIMIT, 1)
    try:
        for _ in range(100):
            attend(K, q, cache, pos, i32([n] * B), 0, qp, B, T, Hq, H, D, so)
            try:
                K.kvc_check_status()
            except K.KvcError as e:
                assert e.code == K.KVC_ERR_TIMEOUT
                gave_up = True
                break
    finally:
        K.kvc_set_option(K.KVC_OPT_WAIT_LIMIT, 0)
    assert gave_up


def test_offsets_past_32_bits_of_many_rows(K):
    """The many-row form at the far end of a slot of 2^25 rows, 4.8 GB."""
    D, cap, T, Hq = 128, 1 << 25, 9, 4
    so = [0, cap]
    cache = torch.zeros(cap * D * 9 // 8, dtype=torch.uint8, device="cuda")
    pos = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    k, v, q = rnd(1, 1, 1, 40, D), rnd(2, 1, 1, 40, D), rnd(3, 1, Hq, T, D)
    rows, qp = i32([[cap - 43]]), 30 + np.arange(T)
    K.kvc_append_q4(k, v, i32([np.arange(40)]), 1, 1, 40, D, so, rows, cache, pos)
    out, lse = attend(K, q, cache, pos, rows, 43, i32([qp]), 1, T, Hq, 1, D, so)
    K.kvc_check_status()
    hk, hv = O.held(f64(k)[0, 0]), O.held(f64(v)[0, 0])
    for h in range(Hq):
        ref, rl, mag = O.attention(f64(q)[0, h], hk, hv, np.arange(40), qp)
        A = float((np.abs(f64(q)[0, h]) @ np.abs(hk).T).max()) / math.sqrt(D)
        tol = 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -11 + A * 2.0 ** -18) * mag + 40 * 2.0 ** -29 * np.abs(hv).max()
        assert np.all(np.abs(f64(out)[0, h] - ref) <= tol)
        assert np.all(np.abs(f64(lse)[0, h] - rl) <= 2.0 ** -18 * A + 2.0 ** -20 * np.abs(rl) + 2.0 ** -20)


def test_calls_at_the_same_time_on_two_streams(K):
    """Calls of every form on two streams at once, each with a workspace of its own, give the bits
    of the calls alone."""
    H, Hq, D, n = 4, 16, 64, [700, 40, 0, 2000]
    so = K.kvc_q4_layout(H, 1 << 20, n, 0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for i, (B, T) in enumerate([(2, 20), (1, 90), (2, 1), (40, 1), (1, 90), (2, 20)]):
        cache, pos, _, _ = filled(K, B, H, D, so, n, 301 + i)
        q, rows, qp = rnd(401 + i, B, Hq, T, D), i32([n] * B), i32(np.full((B, T), 1 << 20))
        args = (q, cache, pos, rows, 0, qp, B, T, Hq, H, D, so)
        jobs.append((args, attend(K, *args), torch.empty_like(q), torch.empty((B, Hq, T), device="cuda"),
                     K.attention_q4_workspace(B, T, Hq, H, D)))
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (args, _, out, lse, ws) in enumerate(jobs):
            K.kvc_attention_q4(*args, out, lse, ws, stream=streams[i % 2])
    torch.cuda.synchronize()
    K.kvc_check_status()
    for args, (o, l), out, lse, _ in jobs:
        assert torch.equal(out, o) and torch.equal(lse, l)


# ------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("B,T", [(2, 1), (40, 1), (1, 20)])
def test_two_graphs_share_a_workspace(K, B, T):
    """Two captured calls over different caches replayed in turn on one stream, on one workspace,
    give what the calls give alone (clusters, ranges, many rows)."""
    H, Hq, D, n = 4, 16, 128, [300, 40, 0, 77]
    so = K.kvc_q4_layout(H, 1000, n, 0)
    ws = K.attention_q4_workspace(B, T, Hq, H, D)
    calls, alone = [], []
    for seed in (201, 301):
        cache, pos, _, _ = filled(K, B, H, D, so, n, seed)
        q, qp, rows = rnd(seed + 1, B, Hq, T, D), i32(np.full((B, T), 5000)), i32([n] * B)
        out, lse = torch.empty_like(q), torch.empty((B, Hq, T), device="cuda")
        args = (q, cache, pos, rows, 0, qp, B, T, Hq, H, D, so)
        alone.append(attend(K, *args))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            K.kvc_attention_q4(*args, out, lse, ws)
        calls.append((graph, out, lse, args))
    for _ in range(3):
        for graph, _, _, _ in calls:
            graph.replay()
    K.kvc_check_status()
    for (_, out, lse, _), (o, l) in zip(calls, alone):
        assert torch.equal(out, o) and torch.equal(lse, l)


def test_another_stream_and_a_replayed_graph(K):
    """A captured decoding step (append, attention) is replayed while the caller's row counts
    grow; it gives what the calls give one by one on another stream."""
    B, H, Hq, D, n = 2, 2, 8, 128, [60, 33]
    so = K.kvc_q4_layout(H, 1000, n, 12)
    steps = [(rnd(100 + i, B, H, 1, D), rnd(200 + i, B, H, 1, D), rnd(300 + i, B, Hq, 1, D)) for i in range(8)]
    results = []
    for captured in (False, True):
        cache, pos, _, _ = filled(K, B, H, D, so, n, 95)
        rows, qp = i32([n, n]), i32([[500], [600]])
        k, v, q = (torch.empty_like(t) for t in steps[0])
        ws = K.attention_q4_workspace(B, 1, Hq, H, D)
        out, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")

        def step():
            K.kvc_append_q4(k, v, qp, B, H, 1, D, so, rows, cache, pos)
            K.kvc_attention_q4(q, cache, pos, rows, 1, qp, B, 1, Hq, H, D, so, out, lse, ws)
            rows.add_(1)
            qp.add_(1)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = []
        with torch.cuda.stream(side):
            graph = None
            for i, (a, b, c) in enumerate(steps):
                k.copy_(a), v.copy_(b), q.copy_(c)
                if captured and graph is None:
                    side.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=side):
                        step()
                if captured:
                    graph.replay()
                else:
                    step()
                got.append((out.clone(), lse.clone()))
        side.synchronize()
        K.kvc_check_status(side)
        assert rows.tolist() == [[68, 41]] * 2
        results.append(got)
    for (a, la), (b, lb) in zip(*results):
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("name,over,K_l", [
    ("tiny", {}, [128, 128]), ("tiny", dict(B=2, S=700, C=700, D=128, H_q=6, pool_k=7, hh_frac=0.03), [90, 333]),
    ("tiny", dict(S=100, C=100), [100, 500]),
])
def test_compress_into_the_4bit_cache(K, name, over, K_l):
    """kvc_compress_layer_q4 keeps what kvc_compress_layer keeps, in 4 bits."""
    cfg = get_config(name, **over)
    inp = make_layer_inputs(cfg)
    q, k, v = inp.q_win.cuda(), inp.k.cuda(), inp.v.cuda()
    B, H, S, D = cfg.B, cfg.H_kv, cfg.S, cfg.D
    ws = K.workspace(B, cfg.H_q, H, D, cfg.W, cfg.b_s, max(K_l), cfg.pool_k)
    head = (cfg.N, 0, B, S, cfg.C, cfg.H_q, H, D, cfg.W, K_l, cfg.sink, cfg.recent, cfg.pool_k, cfg.b_s, q, k, v)
    ko, vo, po, off = K.retained_outputs(B, H, S, D, K_l)
    K.kvc_compress_layer(*head, ko, vo, po, ws)
    so = K.kvc_q4_layout(H, S, K_l, 8)
    ready = torch.cuda.Event()
    ready.record()
    for ev in (None, ready):
        cache, pos = K.q4_cache(B, D, so)
        K.kvc_compress_layer_q4(*head, so, cache, pos, ws, v_ready=ev)
        K.kvc_check_status()
        kk, vv = all_rows(K, cache, B, H, D, so)
        for b in range(B):
            for h in range(H):
                r, n = b * off[-1] + off[h], min(K_l[h], S)
                assert torch.equal(pos.view(B, -1)[b, so[h]:so[h] + n], po[r:r + n])
                assert torch.all(pos.view(B, -1)[b, so[h] + n:so[h + 1]] == -1)
                assert np.array_equal(kk[b, so[h]:so[h] + n], O.held(f64(ko)[r:r + n]))
                assert np.array_equal(vv[b, so[h]:so[h] + n], O.held(f64(vo)[r:r + n]))


def test_prefill_compress_decode(K):
    """The whole use: the prompt's projections are normed and rotated into the active buffers chunk
    by chunk, the layer is compressed into the 4-bit cache, new tokens are decoded over it, and the
    rows read back are what attention saw."""
    B, S, C, Hq, H, D, W = 2, 300, 128, 6, 2, 128, 16
    K_l, T = [64, 100], 3
    ld = (Hq + 2 * H) * D
    inv = (1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    w = (rnd(1, D, scale=0.1) + 1), (rnd(2, D, scale=0.1) + 1)
    k_act, v_act = (torch.zeros((B, H, S, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    prompt = rnd(3, B, S, ld)
    q_all = torch.empty((B, Hq, S, D), dtype=torch.bfloat16, device="cuda")
    split = lambda x: (x[..., :Hq * D], x[..., Hq * D:(Hq + H) * D], x[..., (Hq + H) * D:])
    for c0 in range(0, S, C):
        n = min(C, S - c0)
        part = prompt[:, c0:c0 + n].contiguous()
        pos = torch.arange(c0, c0 + n, dtype=torch.int32, device="cuda").repeat(B, 1)
        qc = torch.empty((B, Hq, n, D), dtype=torch.bfloat16, device="cuda")
        K.kvc_qk_norm_rope(*split(part), B, n, Hq, H, D, ld, ld, ld, D, 0, *w, 1e-6, inv, pos, S, c0, qc, k_act, v_act)
        q_all[:, :, c0:c0 + n] = qc
    q_win = q_all[:, :, S - W:].contiguous()
    so = K.kvc_q4_layout(H, S, K_l, 5 * T)
    cache, pos = K.q4_cache(B, D, so)
    ws = K.workspace(B, Hq, H, D, W, 128, max(K_l), 7)
    K.kvc_compress_layer_q4(1, 0, B, S, C, Hq, H, D, W, K_l, 4, W, 7, 128, q_win, k_act, v_act, so, cache, pos, ws)
    K.kvc_check_status()
    for b in range(B):                       # the selection follows the scores of these keys
        for h in range(H):
            G = Hq // H
            qs = f64(q_win[b, h * G:(h + 1) * G]).reshape(G * W, D)
            s = kvc_oracle.score_head(qs, k_act[b, h].cpu(), W, 7)["s"]
            kept = set(pos.view(B, -1)[b, so[h]:so[h] + K_l[h]].tolist())
            order = np.argsort(-s[4:S - W]) + 4
            sure = order[:K_l[h] - 20]
            cut = s[order[K_l[h] - 21]]
            assert {int(i) for i in sure if s[i] > cut * 1.004} <= kept
    rows = i32([K_l, K_l])
    for step in range(4):
        tok = rnd(10 + step, B, T, ld)
        new = (S + T * step + torch.arange(T, dtype=torch.int32, device="cuda")).repeat(B, 1)
        q, k, v = (torch.empty((B, n, T, D), dtype=torch.bfloat16, device="cuda") for n in (Hq, H, H))
        K.kvc_qk_norm_rope(*split(tok), B, T, Hq, H, D, ld, ld, ld, D, 0, *w, 1e-6, inv, new, T, 0, q, k, v)
        K.kvc_append_q4(k, v, new, B, H, T, D, so, rows, cache, pos)
        args = (q, cache, pos, rows, T, new, B, T, Hq, H, D, so)
        out, lse = attend(K, *args)
        K.kvc_check_status()
        check_attention(K, *args, out, lse)
        ko, vo = (torch.empty((B, H, T, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        K.kvc_read_q4(cache, B, H, D, so, rows, [T] * H, ko, vo)
        assert np.array_equal(f64(ko), O.held(f64(k))) and np.array_equal(f64(vo), O.held(f64(v)))
        rows.add_(T)


def test_tensors_of_another_place_or_kind_are_refused(K):
    D, so = 64, [0, 16]
    cache, pos = K.q4_cache(1, D, so)
    q, out = rnd(1, 1, 2, 1, D), torch.empty((1, 2, 1, D), dtype=torch.bfloat16, device="cuda")
    ws = K.attention_q4_workspace(1, 1, 2, 1, D)
    rows, qp = i32([[1]]), i32([[1]])
    call = lambda **o: K.kvc_attention_q4(**{**dict(q=q, cache=cache, pos=pos, rows=rows, extra=0, q_pos=qp, B=1, T=1,
                                                    H_q=2, H_kv=1, D=D, slot_off=so, out=out, lse=None, ws=ws), **o})
    for bad in (dict(q=q.cpu()), dict(rows=rows.long()), dict(cache=cache[:-1]), dict(out=out.float()),
                dict(q=torch.stack((q, q), -1)[..., 0]), dict(pos=pos[1:]), dict(ws=ws[:256]), dict(ws=ws[1:]),
                dict(ws=ws.cpu()), dict(ws=ws.float())):
        with pytest.raises(K.KvcError):
            call(**bad)
    call()
    K.kvc_check_status()
