"""Attention of a prompt chunk over the active layer's buffers, against the fp64
definition (bounds: attend_util).  Weights are rounded to bf16 (w = 2^-8); queries and
keys are exact."""

import numpy as np
import pytest
import torch

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


def run(K, q, k, v, qp, first, last, S, cap=0.0, slopes=None, lse=True, ws=None, out=None, stream=None):
    B, Hq, T, D = q.shape
    H = k.shape[1]
    if ws is None:
        ws = K.attention_chunk_workspace(B, T, Hq, H, D)
        ws.fill_(0xff)
    if out is None:
        out = torch.full((B, Hq, T, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full((B, Hq, T), float("nan"), device="cuda") if lse else None
    K.kvc_attention_chunk(q, k, v, qp, first, last, B, T, Hq, H, S, D, cap, slopes, out, ls, ws, stream=stream)
    return out, ls


def seen(qp, first, last, S):
    """[B, T, S]"""
    qp = qp.cpu().numpy()
    lo = np.zeros_like(qp) if first is None else first.cpu().numpy()
    hi = qp if last is None else last.cpu().numpy()
    j = np.arange(S)
    return (j >= lo[..., None]) & (j <= hi[..., None]) & (qp >= 0)[..., None]


def verify(q, k, v, qp, first, last, S, cap, slopes, out, lse, heads=None, batches=None):
    B, Hq, T, D = q.shape
    H = k.shape[1]
    see = seen(qp, first, last, S)
    far = np.abs(qp.cpu().numpy()[..., None].astype(np.int64) - np.arange(S))
    qn, kn, vn, on, ln = f64(q), f64(k), f64(v), f64(out), f64(lse)
    sl = np.zeros(Hq) if slopes is None else f64(slopes)
    for b in batches if batches is not None else range(B):
        for hq in heads if heads is not None else range(Hq):
            h = hq // (Hq // H)
            check(qn[b, hq], kn[b, h], vn[b, h], see[b], far[b], cap, sl[hq], on[b, hq], ln[b, hq], 2.0 ** -8, 0.0, 0.0,
                  (b, hq))


def poison(k, v, see):
    """NaN where no query of the call sees."""
    gone = torch.as_tensor(~see.any(1)).cuda()                     # [B, S]
    nan = torch.tensor(float("nan"), dtype=k.dtype, device="cuda")
    return (torch.where(gone[:, None, :, None], nan, x).contiguous() for x in (k, v))


SHAPES = [  # B, T, Hq, H, S, row0, D
    (1, 1, 4, 1, 1, 0, 128),           # one key
    (1, 1, 32, 8, 1000, 999, 128),     # a single token, few rows
    (2, 5, 10, 2, 700, 600, 64),
    (1, 16, 32, 4, 4096, 4080, 128),   # a full tile of rows, key pairs
    (1, 17, 32, 4, 515, 498, 64),      # one token more: row pairs
    (1, 128, 2, 2, 128, 0, 128),       # G = 1
    (3, 129, 3, 1, 300, 150, 64),      # G = 3, ragged tiles
    (1, 257, 7, 1, 513, 256, 128),     # G = 7
    (2, 300, 16, 2, 2048, 1000, 128),
    (1, 33, 128, 1, 640, 600, 64),     # 128 query heads a KV head: a token a tile
]


@pytest.mark.parametrize("B,T,Hq,H,S,row0,D", SHAPES)
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (5.0, True)])
def test_causal(K, B, T, Hq, H, S, row0, D, cap, bias):
    q, k, v = rnd(1, B, Hq, T, D, scale=1.5), rnd(2, B, H, S, D), rnd(3, B, H, S, D)
    qp = i32(np.arange(row0, row0 + T)[None].repeat(B, 0))
    kp, vp = poison(k, v, seen(qp, None, None, S))
    sl = slopes_of(Hq, bias)
    out, lse = run(K, q, kp, vp, qp, None, None, S, cap, sl)
    K.kvc_check_status()
    verify(q, k, v, qp, None, None, S, cap, sl, out, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True), (30.0, True)])
def test_documents_and_padding(K, D, T, cap, bias):
    """Documents, tokens that see nothing among others, keys between documents that no one sees."""
    B, Hq, H, S = 2, 8, 2, 900
    g = np.random.default_rng(D + T)
    q, k, v = rnd(4, B, Hq, T, D, scale=1.5), rnd(5, B, H, S, D), rnd(6, B, H, S, D)
    qp = np.sort(g.choice(S, (B, T)), 1)
    first = qp - g.integers(0, 260, (B, T))
    last = qp + g.integers(-3, 2, (B, T))
    first[:, -1], last[0, 0] = qp[:, -1] + 5, -7                  # empty ranges
    qp[1, T // 2:] = -1
    qp, first, last = i32(qp), i32(first), i32(last)
    kp, vp = poison(k, v, seen(qp, first, last, S))
    sl = slopes_of(Hq, bias)
    out, lse = run(K, q, kp, vp, qp, first, last, S, cap, sl)
    K.kvc_check_status()
    verify(q, k, v, qp, first, last, S, cap, sl, out, lse)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("prefix", [0, 1, 700, 1100, 2000])
def test_prefix(K, prefix, bias):
    """A prefix that ends before, in and behind the chunk; ranges that pass the buffer's end."""
    B, T, Hq, H, S, D, row0 = 1, 256, 4, 2, 1200, 128, 900
    q, k, v = rnd(7, B, Hq, T, D, scale=1.5), rnd(8, B, H, S, D), rnd(9, B, H, S, D)
    qp = i32(np.arange(row0, row0 + T)[None])
    last = torch.clamp(qp, min=prefix - 1).contiguous()
    sl = slopes_of(Hq, bias)
    out, lse = run(K, q, k, v, qp, None, last, S, 0.0, sl)
    K.kvc_check_status()
    verify(q, k, v, qp, None, last, S, 0.0, sl, out, lse)


def test_nothing_is_seen(K):
    B, T, Hq, H, S, D = 2, 70, 8, 4, 300, 64
    q = rnd(1, B, Hq, T, D)
    k = torch.full((B, H, S, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, lse = run(K, q, k, k, i32(np.full((B, T), -1)), None, None, S)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    K.kvc_check_status()


@pytest.mark.parametrize("T", [1, 40, 2048])
def test_many_parts(K, T):
    """Units cut over many ranges, long caches, large scores; heads sampled."""
    B, Hq, H, S, D = 1, 8, 2, 20000, 128
    q, k, v = rnd(11, B, Hq, T, D, scale=4.0), rnd(12, B, H, S, D), rnd(13, B, H, S, D)
    qp = i32(np.arange(S - T, S)[None])
    out, lse = run(K, q, k, v, qp, None, None, S)
    K.kvc_check_status()
    pick = slice(max(0, T - 300), T)
    verify(q[:, :, pick].contiguous(), k, v, qp[:, pick].contiguous(), None, None, S, 0.0, None,
           out[:, :, pick].contiguous(), lse[:, :, pick].contiguous(), heads=[0, 3, 5])


@pytest.mark.parametrize("B,T", [(12, 40), (20, 250), (150, 250), (1100, 250)])
def test_many_units(K, B, T):
    """Few units, which every CTA plans; more; more than the planning kernel counts itself; more than
    its shared memory holds.  And more than ranges, in each."""
    Hq, H, S, D = 6, 2, 260, 64
    q, k, v = rnd(14, B, Hq, T, D), rnd(15, B, H, S, D), rnd(16, B, H, S, D)
    qp = i32(np.random.default_rng(0).integers(-40, 110, (B, 1)) + np.arange(T)[None])
    out, lse = run(K, q, k, v, qp, None, None, S)
    K.kvc_check_status()
    pick = sorted({0, 1, B // 2, B - 2, B - 1})
    at = [x[pick].contiguous() for x in (q, k, v, qp, out, lse)]
    verify(*at[:4], None, None, S, 0.0, None, *at[4:], heads=[1, 4])
    assert torch.isfinite(out).all()


def test_scores_that_grow(K):
    """The reference moves in nearly every tile, up to large scores, and stays there."""
    B, T, Hq, H, S, D = 1, 64, 4, 2, 2048, 128
    q = rnd(17, B, Hq, T, D, scale=3.0)
    k = rnd(18, B, H, S, D)
    k = (k.float() * torch.linspace(0.01, 12, S, device="cuda")[None, None, :, None]).to(torch.bfloat16)
    v = rnd(19, B, H, S, D)
    qp = i32(np.arange(S - T, S)[None])
    out, lse = run(K, q, k, v, qp, None, None, S)
    verify(q, k, v, qp, None, None, S, 0.0, None, out, lse)
    # and falling: the first tile has the largest
    out, lse = run(K, q, k.flip(2).contiguous(), v, qp, None, None, S)
    verify(q, k.flip(2), v, qp, None, None, S, 0.0, None, out, lse)


@pytest.mark.parametrize("cap,scale", [(2.0 ** -20, 1.0), (0.5, 3.0), (10.0, 8.0), (60.0, 3.0)])
def test_cap_of_every_size(K, cap, scale):
    """Scores far below, around and far above the cap."""
    B, T, Hq, H, S, D = 1, 32, 4, 2, 500, 64
    q, k, v = rnd(20, B, Hq, T, D, scale=scale), rnd(21, B, H, S, D), rnd(22, B, H, S, D)
    qp = i32(np.arange(S - T, S)[None])
    out, lse = run(K, q, k, v, qp, None, None, S, cap)
    verify(q, k, v, qp, None, None, S, cap, None, out, lse)
    K.kvc_check_status()


@pytest.mark.parametrize("cap,scale", [(50.0, 0.3), (1.0, 0.02), (2.0 ** -6, 0.0005), (1e4, 1.0), (8.0, 1.0), (4.5, 1.0)])
@pytest.mark.parametrize("S,D", [(130, 128), (1500, 64)])
def test_cap_above_most_scores(K, S, D, cap, scale):
    """Scores below the cap, but for the queries of a few tokens: tiles of each form of the tangent."""
    B, T, Hq, H = 2, 130, 4, 2
    q, k, v = rnd(23, B, Hq, T, D, scale=scale), rnd(24, B, H, S, D), rnd(25, B, H, S, D)
    q[:, 1:, 100:103] *= 32
    qp = i32(np.stack([np.arange(S - T, S)] * B))
    out, lse = run(K, q, k, v, qp, None, None, S, cap)
    verify(q, k, v, qp, None, None, S, cap, None, out, lse)
    K.kvc_check_status()


def test_a_cap_far_above_the_scores_leaves_them(K):
    """The tangent's error is relative to the score: bounds as without a cap of scores below 100."""
    B, T, Hq, H, S, D = 1, 32, 4, 2, 500, 64
    q, k, v = rnd(20, B, Hq, T, D, scale=2.0), rnd(21, B, H, S, D), rnd(22, B, H, S, D)
    qp = i32(np.arange(S - T, S)[None])
    out, lse = run(K, q, k, v, qp, None, None, S, 2.0 ** 20)
    free, free_lse = run(K, q, k, v, qp, None, None, S)
    assert float((lse - free_lse).abs().max()) <= 100 * 2.0 ** -20 + 2.0 ** -18
    verify(q, k, v, qp, None, None, S, 0.0, None, out, free_lse)


def test_no_lse_same_bits_and_streams(K):
    """The same call twice gives the same bits; without lse; on a stream of the caller's."""
    B, T, Hq, H, S, D = 2, 100, 8, 2, 3000, 128
    q, k, v = rnd(23, B, Hq, T, D), rnd(24, B, H, S, D), rnd(25, B, H, S, D)
    qp = i32(np.arange(S - T, S)[None].repeat(B, 0))
    out, lse = run(K, q, k, v, qp, None, None, S)
    again, lse2 = run(K, q, k, v, qp, None, None, S)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    none, _ = run(K, q, k, v, qp, None, None, S, lse=False)
    assert torch.equal(out, none)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other, _ = run(K, q, k, v, qp, None, None, S, stream=st)
    st.synchronize()
    assert torch.equal(out, other)


def test_captured(K):
    """A captured call follows its device-held masks; two captured calls share a workspace."""
    B, T, Hq, H, S, D = 1, 60, 8, 2, 2500, 128
    q, k, v = rnd(26, B, Hq, T, D), rnd(27, B, H, S, D), rnd(28, B, H, S, D)
    qp, first = i32(np.arange(1000, 1000 + T)[None]), i32(np.zeros((B, T)))
    ws = K.attention_chunk_workspace(B, T, Hq, H, D)
    out = torch.empty_like(q)
    two = torch.empty_like(q)
    q2 = rnd(29, B, Hq, T, D)
    run(K, q, k, v, qp, first, None, S, ws=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kvc_attention_chunk(q, k, v, qp, first, None, B, T, Hq, H, S, D, 0.0, None, out, None, ws)
        K.kvc_attention_chunk(q2, k, v, qp, first, None, B, T, Hq, H, S, D, 0.0, None, two, None, ws)
    for at, lo in ((0, 0), (2440, 0), (1500, 1300)):
        qp.copy_(i32(np.arange(at, at + T)[None]))
        first.fill_(lo)
        g.replay()
        want, lse = run(K, q, k, v, qp, first, None, S)
        want2, _ = run(K, q2, k, v, qp, first, None, S)
        assert torch.equal(out, want) and torch.equal(two, want2)
        verify(q, k, v, qp, first, None, S, 0.0, None, want, lse, heads=[0, 7])


def test_offsets_past_32_bits(K):
    """Buffers of 2^32 elements and more: the last head's keys, and queries at the far end of a sequence."""
    B, T, Hq, H, S, D = 1, 3, 3, 3, 12 << 20, 128
    k, v = (torch.zeros((B, H, S, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, tail = rnd(50, B, Hq, T, D, scale=2.0), 300
    k[0, :, S - tail:], v[0, :, S - tail:] = rnd(51, H, tail, D), rnd(52, H, tail, D)
    qp, first = i32([[S - 3, S - 2, S - 1]]), i32([[S - 200, S - 290, S - 1]])
    out, lse = run(K, q, k, v, qp, first, None, S)
    K.kvc_check_status()
    at = S - tail
    verify(q, k[:, :, at:], v[:, :, at:], qp - at, first - at, None, tail, 0.0, None, out, lse)


@pytest.mark.parametrize("mask", ["first", "last"])
def test_steep_and_negative_slopes(K, mask):
    """Slopes from 2^-20 to 8, and negative ones, which favour far keys; keys ahead of the query."""
    B, T, Hq, H, S, D = 1, 70, 8, 2, 1500, 64
    q, k, v = rnd(53, B, Hq, T, D), rnd(54, B, H, S, D), rnd(55, B, H, S, D)
    qp = i32(np.arange(800, 800 + T)[None])
    first, last = (i32(np.arange(300, 300 + T)[None]), None) if mask == "first" else (None, i32(np.full((B, T), 1400)))
    sl = torch.tensor([2.0 ** -20, 2.0 ** -10, 0.01, 0.5, 2.0, 8.0, 0.0, -0.02], device="cuda")
    out, lse = run(K, q, k, v, qp, first, last, S, 0.0, sl)
    K.kvc_check_status()
    verify(q, k, v, qp, first, last, S, 0.0, sl, out, lse)


@pytest.mark.parametrize("level", [-3000.0, -100.0, 100.0, 3000.0])
def test_scores_of_every_level(K, level):
    """Rows whose scores all lie far from the last row's: the reference that a segment starts from is
    another row's, and has to move either way; many segments a range."""
    B, T, Hq, H, S, D = 6, 200, 4, 2, 200, 64
    q, k, v = rnd(56, B, Hq, T, D), rnd(57, B, H, S, D), rnd(58, B, H, S, D)
    q[..., 0] = 8.0
    k[..., 0] = torch.where(torch.arange(B, device="cuda") % 2 == 0, level, -level)[:, None, None].to(torch.bfloat16)
    qp = i32(np.arange(T)[None].repeat(B, 0))
    out, lse = run(K, q, k, v, qp, None, None, S)
    K.kvc_check_status()
    verify(q, k, v, qp, None, None, S, 0.0, None, out, lse, heads=[0, 3])


def test_a_wait_that_gives_up(K):
    """With a limit of one poll a wait may give up: the call ends all the same and says so, a call
    in which none did is right, and so is the next one."""
    B, T, Hq, H, S, D = 4, 64, 32, 8, 6000, 128
    q, k, v = rnd(30, B, Hq, T, D), rnd(31, B, H, S, D), rnd(32, B, H, S, D)
    qp = i32(np.arange(S - T, S)[None].repeat(B, 0))
    want, lse = run(K, q, k, v, qp, None, None, S)
    verify(q, k, v, qp, None, None, S, 0.0, None, want, lse, heads=[0])
    gave_up = False
    K.kvc_set_option(K.KVC_OPT_WAIT_LIMIT, 1)
    try:
        for _ in range(300):
            out, _ = run(K, q, k, v, qp, None, None, S)
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
    out, _ = run(K, q, k, v, qp, None, None, S)
    K.kvc_check_status()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 130])
def test_non_finite_query_stays_in_its_row(K, T):
    B, Hq, H, S, D = 1, 8, 2, 600, 64
    q, k, v = rnd(33, B, Hq, T, D), rnd(34, B, H, S, D), rnd(35, B, H, S, D)
    qp = i32(np.arange(S - T, S)[None])
    want, _ = run(K, q, k, v, qp, None, None, S)
    bad = q.clone()
    bad[0, 2, T - 1, 5] = float("nan")
    out, _ = run(K, bad, k, v, qp, None, None, S)
    assert torch.isnan(out[0, 2, T - 1]).all()
    out[0, 2, T - 1] = want[0, 2, T - 1]
    assert torch.equal(out, want)
