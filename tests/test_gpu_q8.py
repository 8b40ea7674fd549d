"""The 8-bit retained cache and attention over it, against the fp64 definition.

The cache's values are compared exactly: scales are powers of two and codes roundings
of exact quotients.  Attention bounds: attend_util, with the weights' and queries'
roundings of the two forms: up to 8 query rows per KV head fp16 (w = 2^-11; weights
below fp16's normal numbers half a step, 2^-25, where the largest is at least 2^4 less the
values' scales, which the blocks of normal values here leave within 2^4 of one
another: floor = 2^-25; queries 2^-24 of the row's largest), more rows two e4m3
parts (w = 2^-8: the first is cut to 4 significant bits, the rest, at most 2^-3 of the
weight, is rounded to 4 of its own, half a step of which is 2^-8 of the weight's binade;
floor: half of e4m3's smallest step, 2^-10, where the row's largest weight is at least
2^5, so 2^-15, and by the same scales 2^-11; queries 2^-17)."""

import math

import numpy as np
import pytest
import torch

from oracle import serve as O
from synth import get_config, make_layer_inputs
from tests.attend_util import check, f64, i32, rnd, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_score_kv_gb300 import build
    build.build()
    import attention_score_kv_gb300.kvc as kvc
    return kvc


def read_all(K, c, B, H, D, so):
    n = [so[h + 1] - so[h] for h in range(H)]
    k, v = (torch.empty((B * so[H], D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K.kvc_read_q8(*c[:3], B, H, D, so, None, n, k, v, out_off=list(so))
    return f64(k).reshape(B, so[H], D), f64(v).reshape(B, so[H], D)


def empty_cache(K, B, D, so, byte=0xff):
    """A cache whose bytes are all NaN codes and NaN scales."""
    c = K.q8_cache(B, D, so)
    c[0].fill_(byte), c[1].fill_(byte), c[2].fill_(float("nan"))
    return c


def filled(K, B, H, D, so, n, seed, scale=1.0):
    S = max(max(n), 1) * 3
    k, v = rnd(seed, B, H, S, D, scale=scale), rnd(seed + 1, B, H, S, D)
    c = empty_cache(K, B, D, so)
    idx = torch.full_like(c[3], -1).view(B, -1)
    for h in range(H):
        idx[:, so[h]:so[h] + n[h]] = torch.arange(n[h], device="cuda", dtype=torch.int32) * 3 % S
    K.kvc_gather_q8(k, v, idx, B, H, S, D, n, so, *c)
    return c, k, v


# ------------------------------------------------------------------ the rows
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shift", [0, 8])
def test_values_of_every_kind(K, D, shift):
    """Every exponent, significands around 448's, borders between codes, subnormal codes;
    tensors that start on 32 bytes and on 16."""
    S = 1024
    x = rnd(5, S, D).float()
    for i in range(32):                     # a block each: exponents of largest values from 2^-120 to 2^127
        x[16 * i:16 * i + 16] *= 2.0 ** (i * 8 - 122)
    for i in range(16):                     # largest values around 448 * 2^k, and a spread of 2^0 .. 2^-20 below
        blk = x[512 + 16 * i:528 + 16 * i]
        blk *= torch.exp2(-torch.arange(16, device="cuda") * 1.25)[:, None]
        blk[0, 0] = (1.75 + (i - 8) / 128) * 2.0 ** (i - 5)
        blk[0, 1:] = blk[0, 1:].clamp(-1, 1) * 2.0 ** (i - 6)
    grid = torch.tensor([(8 + i / 2) / 8 for i in range(16)], device="cuda")      # codes and the ties between them
    x[768:784] = (grid.repeat(D // 16) * torch.exp2(torch.arange(16, device="cuda") - 12.0)[:, None]).flip(0)
    x[784] = 0
    x[800:816] = 0                          # a block of zeros
    x[816:832] = 1e-38
    x[832, 0] = 3.38e38
    x = x.to(torch.bfloat16)
    buf = torch.zeros(S * D + 16, dtype=torch.bfloat16, device="cuda")
    a = buf[shift:shift + S * D].view(1, 1, S, D).copy_(x.view(1, 1, S, D))
    y = x.flip(0).contiguous().view(1, 1, S, D)
    so = K.kvc_q4_layout(1, S, [S], 0)
    c = empty_cache(K, 1, D, so)
    K.kvc_gather_q8(a, y, torch.arange(S, dtype=torch.int32, device="cuda"), 1, 1, S, D, [S], so, *c)
    k, v = read_all(K, c, 1, 1, D, so)
    K.kvc_check_status()
    (hk, sk), (hv, sv) = O.held8(f64(x)), O.held8(f64(y)[0, 0])
    assert np.array_equal(f64(c[2]), np.stack((sk, sv), 1))
    assert np.array_equal(k[0], hk) and np.array_equal(v[0], hv)
    assert torch.equal(c[3], torch.arange(S, dtype=torch.int32, device="cuda"))
    # the codes are plain e4m3 rows
    codes = c[0].view(torch.float8_e4m3fn).double().cpu().numpy().reshape(-1, 16, D)
    assert np.array_equal((codes * sk[:, None, None]).reshape(S, D), hk)


@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_not_finite(K, D):
    x = rnd(6, 1, 1, 48, D)
    x[0, 0, 1, 3], x[0, 0, 18, 17], x[0, 0, 19, 60] = float("nan"), float("inf"), float("-inf")
    so = [0, 48]
    c = empty_cache(K, 1, D, so)
    K.kvc_gather_q8(x, x, torch.arange(48, dtype=torch.int32, device="cuda"), 1, 1, 48, D, [48], so, *c)
    with pytest.raises(K.KvcError) as e:
        K.kvc_check_status()
    assert e.value.code == K.KVC_ERR_DEVICE
    k, v = read_all(K, c, 1, 1, D, so)
    want, _ = O.held8(f64(x)[0, 0])
    assert np.array_equal(k[0], want) and np.array_equal(v[0], want) and np.isfinite(want).all()


@pytest.mark.parametrize("D", [64, 128])
def test_gather_of_uneven_heads(K, D):
    """Budgets of 0, 1, 15, 16, 17 and above S; rows behind the last block are left."""
    B, S = 2, 300
    n = [0, 1, 15, 16, 17, 400]
    H = len(n)
    so = K.kvc_q4_layout(H, S, n, 20)
    k, v = rnd(7, B, H, S, D), rnd(8, B, H, S, D)
    c = empty_cache(K, B, D, so, 0x55)
    c[2].fill_(2.0)
    c[3].fill_(-9)
    idx = torch.full((B, so[H]), -1, dtype=torch.int32)
    g = np.random.default_rng(1)
    kept = [min(x, S) for x in n]
    for b in range(B):
        for h in range(H):
            idx[b, so[h]:so[h] + kept[h]] = torch.as_tensor(np.sort(g.permutation(S)[:kept[h]]))
    K.kvc_gather_q8(k, v, idx.cuda(), B, H, S, D, n, so, *c)
    K.kvc_check_status()
    kk, vv = read_all(K, c, B, H, D, so)
    kn, vn = f64(k), f64(v)
    pos = c[3].view(B, -1).cpu().numpy()
    raw = c[0].view(B, so[H], D).cpu().numpy()
    for b in range(B):
        for h in range(H):
            at = idx[b, so[h]:so[h] + kept[h]].numpy()
            for got, x in ((kk, kn), (vv, vn)):
                assert np.array_equal(got[b, so[h]:so[h] + kept[h]], O.held8(x[b, h, at])[0])
            end = so[h] + (kept[h] + 15) // 16 * 16
            assert np.array_equal(pos[b, so[h]:so[h] + kept[h]], at) and np.all(pos[b, so[h] + kept[h]:so[h + 1]] == -9)
            assert np.all(kk[b, so[h] + kept[h]:end] == 0) and np.all(raw[b, end:so[h + 1]] == 0x55)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 5, 16, 33])
@pytest.mark.parametrize("grow", [0.25, 1.0, 40.0, 2.0 ** 60])
def test_append(K, D, T, grow):
    """New rows at every place in a block, smaller, like and larger than what is held; twice over."""
    n0s = [0, 1, 7, 15, 16, 30, 47]
    H, B, S = len(n0s), 2, 64
    so = K.kvc_q4_layout(H, S, n0s, 60)
    k, v = rnd(9, B, H, S, D), rnd(10, B, H, S, D)
    c = empty_cache(K, B, D, so, 0x33)
    idx = torch.arange(S, dtype=torch.int32, device="cuda").repeat(B * (so[H] // S + 1))[:B * so[H]].contiguous()
    for h in range(H):
        idx.view(B, -1)[:, so[h]:so[h] + n0s[h]] = torch.arange(n0s[h], dtype=torch.int32, device="cuda")
    K.kvc_gather_q8(k, v, idx, B, H, S, D, n0s, so, *c)
    nk, nv = rnd(11, B, H, T, D, scale=grow), rnd(12, B, H, T, D, scale=grow)
    rows = i32(np.array([n0s] * B))
    new = i32(np.arange(1000, 1000 + T)[None].repeat(B, 0))
    for _ in range(2):
        K.kvc_append_q8(nk, nv, new, B, H, T, D, so, rows, *c)
        K.kvc_check_status()
        kk, vv = read_all(K, c, B, H, D, so)
        sc, pos = f64(c[2]).reshape(B, -1, 2), c[3].view(B, -1).cpu().numpy()
        for b in range(B):
            for h, n0 in enumerate(n0s):
                for i, (got, x, y) in enumerate(((kk, k, nk), (vv, v, nv))):
                    held, s = O.held8(f64(x)[b, h, :n0])
                    want, ws = O.append8(held, s, f64(y)[b, h])
                    assert np.array_equal(got[b, so[h]:so[h] + n0 + T], want), (b, h)
                    assert np.array_equal(sc[b, so[h] // 16:so[h] // 16 + len(ws), i], ws), (b, h)
                assert np.array_equal(pos[b, so[h] + n0:so[h] + n0 + T], np.arange(1000, 1000 + T))
                # nothing behind them but the codes of their own block's zeros
                raw = c[0].view(B, so[H], D)[b, so[h] + n0 + T:so[h + 1]].cpu().numpy()
                edge = max(0, (n0 + 15) // 16 * 16 - (n0 + T))
                assert np.all(raw[edge:] == 0x33)


@pytest.mark.parametrize("D", [64, 128])
def test_append_of_absent_tokens_and_without_room(K, D):
    B, H, T = 3, 2, 4
    so = [0, 32, 64]
    c = empty_cache(K, B, D, so)
    c[3].fill_(-1)
    k, v = rnd(13, B, H, T, D), rnd(14, B, H, T, D)
    k[:, :, 2] = float("nan")                                     # an absent token may hold anything
    v[:, :, 2] = float("inf")
    new = i32([[5, 6, -1, 7], [5, 6, -3, 7], [1, 2, -1, 3]])
    before = [t.clone() for t in c]
    K.kvc_append_q8(k, v, new, B, H, T, D, so, i32([[0, 20], [3, 29], [-1, 40]]), *c)
    with pytest.raises(K.KvcError):
        K.kvc_check_status()
    pos = c[3].view(B, -1).cpu().numpy()
    kk, vv = read_all(K, c, B, H, D, so)
    for b, h, n0 in ((0, 0, 0), (0, 1, 20), (1, 0, 3)):
        at = so[h] + n0
        assert pos[b, at:at + 4].tolist() == [int(x) if x >= 0 else -1 for x in new[b].tolist()]
        assert np.all(kk[b, at + 2] == 0) and np.all(vv[b, at + 2] == 0)
    for b, h in ((1, 1), (2, 0), (2, 1)):                         # no room: left as it was
        sl = slice(b * 64 + so[h], b * 64 + so[h + 1])
        for i in (0, 1, 3):
            assert torch.equal(c[i][sl], before[i][sl])


def test_read_of_a_part(K):
    B, H, D = 2, 3, 128
    n = [40, 5, 70]
    so = K.kvc_q4_layout(H, 100, n, 10)
    c, _, _ = filled(K, B, H, D, so, n, 15)
    kk, vv = read_all(K, c, B, H, D, so)
    first, cnt = [[3, 0, 65], [20, 4, 0]], [20, 1, 5]
    off = [0, 22, 30, 40]
    k, v = (torch.full((B * 40, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K.kvc_read_q8(*c[:3], B, H, D, so, i32(first), cnt, k, v, out_off=off)
    K.kvc_check_status()
    for got, want in ((k, kk), (v, vv)):
        got = f64(got).reshape(B, 40, D)
        rest = np.ones((B, 40), bool)
        for b in range(B):
            for h in range(H):
                assert np.array_equal(got[b, off[h]:off[h] + cnt[h]],
                                      want[b, so[h] + first[b][h]:so[h] + first[b][h] + cnt[h]])
                rest[b, off[h]:off[h] + cnt[h]] = False
        assert np.all(got[rest] == 7)
    K.kvc_read_q8(*c[:3], B, H, D, so, i32([[-3, 0, 0], [0, 15, 0]]), cnt, k, v, out_off=off)
    with pytest.raises(K.KvcError):
        K.kvc_check_status()
    assert np.all(f64(k).reshape(B, 40, D)[0, :3] == 0)


def test_compress_into_the_cache(K):
    """The compress into 8-bit rows holds what the compress into bf16 rows gathers."""
    cfg = get_config("tiny", pool_k=7, hh_frac=0.02)
    inp = make_layer_inputs(cfg)
    q, k, v = inp.q_win.cuda(), inp.k.cuda(), inp.v.cuda()
    K_l = [100, 140]
    ws = K.workspace(cfg.B, cfg.H_q, cfg.H_kv, cfg.D, cfg.W, cfg.b_s, max(K_l), cfg.pool_k)
    ko, vo, pos, off = K.retained_outputs(cfg.B, cfg.H_kv, cfg.S, cfg.D, K_l)
    args = (cfg.N, 0, cfg.B, cfg.S, cfg.C, cfg.H_q, cfg.H_kv, cfg.D, cfg.W, K_l, cfg.sink, cfg.recent, cfg.pool_k,
            cfg.b_s, q, k, v)
    K.kvc_compress_layer(*args, ko, vo, pos, ws)
    so = K.kvc_q4_layout(cfg.H_kv, cfg.S, K_l, 30)
    c = empty_cache(K, cfg.B, cfg.D, so)
    K.kvc_compress_layer_q8(*args, so, *c, ws)
    K.kvc_check_status()
    kk, vv = read_all(K, c, cfg.B, cfg.H_kv, cfg.D, so)
    for h in range(cfg.H_kv):
        n = K_l[h]
        assert torch.equal(c[3][so[h]:so[h] + n], pos[off[h]:off[h + 1]])
        assert np.array_equal(kk[0, so[h]:so[h] + n], O.held8(f64(ko[off[h]:off[h + 1]]))[0])
        assert np.array_equal(vv[0, so[h]:so[h] + n], O.held8(f64(vo[off[h]:off[h + 1]]))[0])


# ------------------------------------------------------------------ attention
def attend(K, q, c, rows, extra, qp, H, so, cap=0.0, slopes=None, lse=True, ws=None, out=None, stream=None):
    B, Hq, T, D = q.shape
    if ws is None:
        ws = K.attention_q8_workspace(B, T, Hq, H, D)
        ws.fill_(0xff)
    if out is None:
        out = torch.full((B, Hq, T, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full((B, Hq, T), float("nan"), device="cuda") if lse else None
    K.kvc_attention_q8(q, *c, rows, extra, qp, B, T, Hq, H, D, so, cap, slopes, out, ls, ws, stream=stream)
    return out, ls


def verify(K, q, c, rows, extra, qp, H, so, cap, slopes, out, lse, heads=None):
    B, Hq, T, D = q.shape
    few = Hq // H * T <= 8
    kk, vv = read_all(K, c, B, H, D, so)
    K_pos, rows, qp = (t.cpu().numpy() for t in (c[3].view(B, -1), rows.view(B, H), qp.view(B, T)))
    qn, on, ln = f64(q), f64(out), f64(lse)
    sl = np.zeros(Hq) if slopes is None else f64(slopes)
    for b in range(B):
        for hq in heads if heads is not None else range(Hq):
            h = hq // (Hq // H)
            n = min(max(int(rows[b, h]) + extra, 0), so[h + 1] - so[h])
            p = K_pos[b, so[h]:so[h] + n].astype(np.int64)
            see = (p >= 0) & (p <= qp[b][:, None])
            check(qn[b, hq], kk[b, so[h]:so[h] + n], vv[b, so[h]:so[h] + n], see, qp[b][:, None].astype(np.int64) - p,
                  cap, sl[hq], on[b, hq], ln[b, hq], 2.0 ** -11 if few else 2.0 ** -8, 2.0 ** -25 if few else 2.0 ** -11,
                  2.0 ** -24 if few else 2.0 ** -17, (b, hq))


CALLS = [  # B, T, Hq, H, D, rows per head, extra room
    (1, 1, 1, 1, 128, [1]),
    (1, 1, 4, 1, 64, [0]),
    (2, 1, 32, 8, 128, [1000, 17, 16, 15, 1, 129, 128, 0]),
    (1, 1, 40, 8, 64, [300, 2000, 5, 40, 900, 0, 127, 600]),
    (3, 2, 8, 2, 128, [513, 700]),             # 8 query rows: the last of the few
    (1, 3, 6, 2, 64, [200, 333]),              # 9: the first of the many
    (2, 5, 20, 4, 128, [900, 0, 3, 128]),
    (1, 16, 32, 4, 128, [2000, 100, 1, 640]),  # a whole row tile
    (1, 17, 32, 4, 64, [2000, 100, 1, 640]),
    (2, 100, 14, 2, 128, [700, 33]),
    (1, 300, 8, 8, 64, [100, 200, 300, 0, 16, 1, 1024, 5]),
    (64, 1, 16, 2, 128, [40, 25]),
    (40, 9, 4, 2, 64, [60, 90]),
]


@pytest.mark.parametrize("B,T,Hq,H,D,n", CALLS)
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (5.0, True)])
def test_attention(K, B, T, Hq, H, D, n, cap, bias):
    """New tokens over a cache whose unheld bytes are NaN, among them causal, with holes in it."""
    so = K.kvc_q4_layout(H, 1 << 20, n, T + 5)
    c, _, _ = filled(K, B, H, D, so, n, 20)
    S = max(max(n), 1) * 3
    pos = c[3].view(B, -1)
    if max(n) > 20:                                               # holes: rows that no query sees
        for h in range(H):
            pos[:, so[h] + 3:so[h] + min(n[h], 9)] = -1
    rows = i32(np.array([n] * B))
    qp = i32(np.arange(S, S + T)[None].repeat(B, 0))
    k, v = rnd(22, B, H, T, D), rnd(23, B, H, T, D)
    K.kvc_append_q8(k, v, qp, B, H, T, D, so, rows, *c)
    q = rnd(24, B, Hq, T, D, scale=1.5)
    sl = slopes_of(Hq, bias)
    out, lse = attend(K, q, c, rows, T, qp, H, so, cap, sl)
    K.kvc_check_status()
    verify(K, q, c, rows, T, qp, H, so, cap, sl, out, lse)


@pytest.mark.parametrize("T", [1, 4, 60])
def test_queries_that_see_little(K, T):
    """Queries before every row, between them, behind all; absent tokens; no rows at all."""
    B, Hq, H, D = 3, 8, 2, 128
    n = [300, 200]
    so = K.kvc_q4_layout(H, 1 << 20, n, 0)
    c, _, _ = filled(K, B, H, D, so, n, 25)
    qp = np.random.default_rng(T).integers(-5, 950, (B, T))
    qp[0, 0], qp[1, -1] = -1, 0
    qp = i32(qp)
    rows = i32([[300, 200], [0, 1], [299, 0]])
    q = rnd(26, B, Hq, T, D)
    for cap, bias in ((0.0, False), (0.0, True), (8.0, False)):
        sl = slopes_of(Hq, bias)
        out, lse = attend(K, q, c, rows, 0, qp, H, so, cap, sl)
        K.kvc_check_status()
        verify(K, q, c, rows, 0, qp, H, so, cap, sl, out, lse)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_scales_far_apart(K, T):
    """Blocks whose keys and values differ by powers of two, growing and falling: checked
    against the values' own magnitude, block by block of output share."""
    B, Hq, H, D, N = 1, 8, 2, 64, 640
    so = [0, N, 2 * N]
    g = torch.exp2(torch.linspace(-8, 8, N, device="cuda"))[None, None, :, None]
    k = (rnd(27, B, H, N, D).float() * g.flip(2) * 2.0 ** -8).to(torch.bfloat16)
    q = rnd(29, B, Hq, T, D)
    idx = torch.arange(N, dtype=torch.int32, device="cuda").repeat(2)
    rows, qp = i32([[N, N]]), i32(np.arange(N, N + T)[None])
    few = 4 * T <= 8
    for up in (g, g.flip(2)):
        v = (rnd(28, B, H, N, D).float() * up).to(torch.bfloat16)
        c = empty_cache(K, B, D, so)
        K.kvc_gather_q8(k, v, idx, B, H, N, D, [N, N], so, *c)
        out, lse = attend(K, q, c, rows, 0, qp, H, so)
        kk, vv = read_all(K, c, B, H, D, so)
        for hq in range(Hq):
            h = hq // 4
            sl = slice(so[h], so[h + 1])
            # floor: 2^-25 or 2^-15 of the largest weight times the largest scale, which vmax stands for
            check(f64(q)[0, hq], kk[0, sl], vv[0, sl], np.ones((T, N), bool), None, 0.0, 0.0, f64(out)[0, hq],
                  f64(lse)[0, hq], 2.0 ** -11 if few else 2.0 ** -8, 2.0 ** -25 if few else 2.0 ** -15,
                  2.0 ** -24 if few else 2.0 ** -17, hq)


@pytest.mark.parametrize("T", [1, 20])
def test_far_positions_and_steep_slopes(K, T):
    """Positions up to 2^24 apart, slopes from 2^-20 to 4: rows far behind must not blur near ones."""
    B, Hq, H, D, N = 1, 8, 2, 128, 900
    so = K.kvc_q4_layout(H, N, [N, N], 0)
    k, v = rnd(30, B, H, N, D), rnd(31, B, H, N, D)
    c = empty_cache(K, B, D, so)
    at = np.concatenate((np.arange(300), 5_000_000 + np.arange(300), (1 << 24) - 400 + np.arange(300)))
    K.kvc_gather_q8(k, v, i32(np.concatenate([np.pad(np.arange(N), (0, so[1] - N), constant_values=-1)] * 2)), B, H, N,
                    D, [N, N], so, *c)
    c[3].copy_(i32(np.concatenate([np.pad(at, (0, so[1] - N), constant_values=-1)] * 2)))
    rows, qp = i32([[N, N]]), i32((1 << 24) - 100 + np.arange(T)[None])
    sl = torch.tensor([2.0 ** -20, 2.0 ** -18, 2.0 ** -12, 0.001, 0.3, 1.0, 4.0, 0.0], device="cuda")
    q = rnd(32, B, Hq, T, D)
    out, lse = attend(K, q, c, rows, 0, qp, H, so, 0.0, sl)
    K.kvc_check_status()
    verify(K, q, c, rows, 0, qp, H, so, 0.0, sl, out, lse)


@pytest.mark.parametrize("T", [1, 12])
def test_counts_outside_the_slot(K, T):
    B, Hq, H, D = 1, 8, 2, 64
    so = [0, 64, 128]
    c, _, _ = filled(K, B, H, D, so, [64, 64], 33)
    q = rnd(34, B, Hq, T, D)
    qp = i32(np.full((B, T), 1000))
    out, lse = attend(K, q, c, i32([[200, -4]]), 0, qp, H, so)
    with pytest.raises(K.KvcError):
        K.kvc_check_status()
    verify(K, q, c, i32([[64, 0]]), 0, qp, H, so, 0.0, None, out, lse)


@pytest.mark.parametrize("T", [1, 30])
def test_a_step_captured_and_replayed(K, T):
    """Append and attention of a step as one graph while the cache grows, two attentions with one
    workspace in it; against eager calls, bit by bit."""
    B, Hq, H, D, n = 2, 16, 4, 128, [500, 100, 30, 700]
    so = K.kvc_q4_layout(H, 1 << 20, n, 4 * T)
    c, _, _ = filled(K, B, H, D, so, n, 35)
    c2 = tuple(t.clone() for t in c)
    rows, qp = i32([n] * B), i32(np.arange(5000, 5000 + T)[None].repeat(B, 0))
    k, v, q = torch.empty((B, H, T, D), dtype=torch.bfloat16, device="cuda"), None, rnd(36, B, Hq, T, D)
    v = torch.empty_like(k)
    ws = K.attention_q8_workspace(B, T, Hq, H, D)
    out, two = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty((B, Hq, T), device="cuda")
    sl = slopes_of(Hq, True)

    def step(c, out, two, lse, ws):
        K.kvc_append_q8(k, v, qp, B, H, T, D, so, rows, *c)
        K.kvc_attention_q8(q, *c, rows, T, qp, B, T, Hq, H, D, so, 0.0, None, out, lse, ws)
        K.kvc_attention_q8(q, *c, rows, T, qp, B, T, Hq, H, D, so, 25.0, sl, two, None, ws)

    k.copy_(rnd(40, *k.shape)), v.copy_(rnd(41, *k.shape))
    warm = tuple(t.clone() for t in c)
    step(warm, out, two, lse, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c, out, two, lse, ws)
    for i in range(3):
        k.copy_(rnd(50 + i, *k.shape, scale=2.0 ** i)), v.copy_(rnd(60 + i, *k.shape, scale=2.0 ** i))
        g.replay()
        o2, t2, l2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(lse)
        step(c2, o2, t2, l2, K.attention_q8_workspace(B, T, Hq, H, D).fill_(0xff))
        assert torch.equal(out, o2) and torch.equal(two, t2) and torch.equal(lse, l2)
        assert all(torch.equal(a, b) for a, b in zip(c[:2] + c[3:], c2[:2] + c2[3:]))
        verify(K, q, c, rows, T, qp, H, so, 0.0, None, out, lse, heads=[0, 5, 15])
        rows += T
        qp += T
    K.kvc_check_status()


@pytest.mark.parametrize("T", [1, 24])
def test_two_streams_at_once(K, T):
    """Calls on two streams with workspaces of their own, and a call on no default stream."""
    B, Hq, H, D, n = 4, 16, 4, 64, [900, 1200, 1000, 800]
    so = K.kvc_q4_layout(H, 1 << 20, n, 0)
    c, _, _ = filled(K, B, H, D, so, n, 42)
    rows, qp = i32([n] * B), i32(np.full((B, T), 1 << 20))
    qs = [rnd(43 + i, B, Hq, T, D) for i in range(2)]
    want = [attend(K, q, c, rows, 0, qp, H, so)[0] for q in qs]
    torch.cuda.synchronize()
    sts = [torch.cuda.Stream() for _ in qs]
    ws = [K.attention_q8_workspace(B, T, Hq, H, D) for _ in qs]
    got = [torch.empty_like(q) for q in qs]
    for _ in range(10):
        for i, st in enumerate(sts):
            K.kvc_attention_q8(qs[i], *c, rows, 0, qp, B, T, Hq, H, D, so, 0.0, None, got[i], None, ws[i], stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 9])
def test_offsets_past_32_bits(K, T):
    """A slot of 2^25 rows, 8.6 GB: append and both forms of the attention at its far end."""
    D, cap, Hq = 128, 1 << 25, 4
    so = [0, cap]
    c = (torch.zeros((cap, D), dtype=torch.uint8, device="cuda"), torch.zeros((cap, D), dtype=torch.uint8, device="cuda"),
         torch.ones((cap // 16, 2), device="cuda"), torch.full((cap,), -1, dtype=torch.int32, device="cuda"))
    k, v, q = rnd(1, 1, 1, 40, D), rnd(2, 1, 1, 40, D), rnd(3, 1, Hq, T, D)
    rows, qp = i32([[cap - 43]]), i32([30 + np.arange(T)])
    K.kvc_append_q8(k, v, i32([np.arange(40)]), 1, 1, 40, D, so, rows, *c)
    out, lse = attend(K, q, c, rows, 43, qp, 1, so)
    K.kvc_check_status()
    n = 48                                                        # the slot's last rows, as a cache of their own
    tail = tuple(t[cap - n:].contiguous() for t in c[:2]) + (c[2][-n // 16:].contiguous(), c[3][cap - n:].contiguous())
    few = T == 1
    kk, vv = read_all(K, tail, 1, 1, D, [0, n])
    p = tail[3].cpu().numpy().astype(np.int64)
    see = (p >= 0) & (p <= qp.cpu().numpy()[0][:, None])
    for hq in range(Hq):
        check(f64(q)[0, hq], kk[0], vv[0], see, None, 0.0, 0.0, f64(out)[0, hq], f64(lse)[0, hq],
              2.0 ** -11 if few else 2.0 ** -8, 2.0 ** -25 if few else 2.0 ** -11, 2.0 ** -24 if few else 2.0 ** -17, hq)


@pytest.mark.parametrize("T", [1, 20])
def test_neighbours_may_hold_anything(K, T):
    """Rows of other sequences' slots, of unheld blocks and of tokens that come later in the call are
    NaN codes with NaN and infinite scales; slots without rows; uneven sequences."""
    B, Hq, H, D = 3, 8, 2, 64
    so = [0, 160, 176]
    c = empty_cache(K, B, D, so)
    c[2][::3] = float("inf")
    c[3].fill_(5)                                                 # stale positions
    n = np.array([[130, 0], [0, 16], [7, 3]])
    k, v = rnd(70, B, H, 160, D), rnd(71, B, H, 160, D)
    for b in range(B):
        for h in range(H):
            m = int(n[b, h])
            if not m:
                continue
            part = tuple(t.view(B, -1, *t.shape[1:])[b] for t in c)
            sub = tuple(t.contiguous() for t in part)
            K.kvc_append_q8(k[b:b + 1, :, :m].contiguous(), v[b:b + 1, :, :m].contiguous(), i32([np.arange(m)]), 1, H, m,
                            D, so, i32([[0 if x == h else 1 << 20 for x in range(H)]]), *sub)
            with pytest.raises(K.KvcError):                       # the other head has no room: left as it was
                K.kvc_check_status()
            for t, x in zip(part, sub):
                t.copy_(x)
    q, qp = rnd(72, B, Hq, T, D), i32(np.sort(np.random.default_rng(5).integers(0, 140, (B, T)), 1))
    out, lse = attend(K, q, c, i32(n), 0, qp, H, so)
    K.kvc_check_status()
    verify(K, q, c, i32(n), 0, qp, H, so, 0.0, None, out, lse)


def test_a_wait_that_gives_up(K):
    """With a limit of one poll a wait may give up: the call ends all the same and says so, a call
    in which none did is right, and so is the next one."""
    B, T, Hq, H, D, n = 4, 40, 32, 8, 128, [6000] * 8
    so = K.kvc_q4_layout(H, 1 << 20, n, 0)
    c, _, _ = filled(K, B, H, D, so, n, 44)
    rows, qp, q = i32([n] * B), i32(np.full((B, T), 1 << 20)), rnd(45, B, Hq, T, D)
    want, lse = attend(K, q, c, rows, 0, qp, H, so)
    gave_up = False
    K.kvc_set_option(K.KVC_OPT_WAIT_LIMIT, 1)
    try:
        for _ in range(300):
            out, _ = attend(K, q, c, rows, 0, qp, H, so)
            try:
                K.kvc_check_status()
                assert torch.equal(out, want)
            except K.KvcError as e:
                assert e.code == K.KVC_ERR_TIMEOUT
                gave_up = True
                break
    finally:
        K.kvc_set_option(K.KVC_OPT_WAIT_LIMIT, 0)
    assert gave_up
    out, _ = attend(K, q, c, rows, 0, qp, H, so)
    K.kvc_check_status()
    assert torch.equal(out, want)


def test_a_layer_from_prompt_to_decoding(K):
    """Chunk attention, compress into the 8-bit cache, append, attention over it, in a run; and the
    attention over the cache is the prompt's own where the budget keeps every row."""
    B, Hq, H, D, S, C = 1, 8, 2, 64, 256, 128
    k, v = rnd(46, B, H, S, D), rnd(47, B, H, S, D)
    q = rnd(48, B, Hq, S, D)
    outs = []
    for j in range(S // C):
        qc = q[:, :, j * C:(j + 1) * C].contiguous()
        qp = i32(np.arange(j * C, (j + 1) * C)[None])
        o = torch.empty_like(qc)
        K.kvc_attention_chunk(qc, k, v, qp, None, None, B, C, Hq, H, S, D, 0.0, None, o, None,
                              K.attention_chunk_workspace(B, C, Hq, H, D))
        outs.append(o)
    whole = torch.cat(outs, 2)
    W, K_l = 16, [S, S]
    ws = K.workspace(B, Hq, H, D, W, 128, S, 1)
    so = K.kvc_q4_layout(H, S, K_l, 16)
    c = empty_cache(K, B, D, so)
    K.kvc_compress_layer_q8(1, 0, B, S, C, Hq, H, D, W, K_l, 4, W, 1, 128, q[:, :, S - W:].contiguous(), k, v, so, *c,
                            ws)
    rows = i32([K_l])
    qp = i32(np.arange(S - W, S)[None])
    out, lse = attend(K, q[:, :, S - W:].contiguous(), c, rows, 0, qp, H, so)
    K.kvc_check_status()
    verify(K, q[:, :, S - W:].contiguous(), c, rows, 0, qp, H, so, 0.0, None, out, lse)
    # 4 significant bits a value, averaged over tens of rows: a few parts in a hundred
    a, b = f64(whole[:, :, S - W:]), f64(out)
    assert np.linalg.norm(a - b) <= 2.0 ** -4 * math.sqrt(2) * np.linalg.norm(a)
