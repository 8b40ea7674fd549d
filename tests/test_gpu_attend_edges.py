"""Edges of the attentions on the tensor cores (a prompt chunk's, and the 8-bit cache's with
many query rows) that go across their warps, streams and segments.  Bounds: attend_util,
and those written beside a test."""

import numpy as np
import pytest
import torch

from tests import test_gpu_chunk as C
from tests import test_gpu_q8 as Q
from tests.attend_util import i32, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_score_kv_gb300 import build
    build.build()
    import attention_score_kv_gb300.kvc as kvc
    return kvc


# ------------------------------------------------------- scores that are taken a second time
@pytest.mark.parametrize("T", [40, 200])                           # key pairs, row pairs
@pytest.mark.parametrize("cap", [0.0, 300.0])
def test_moving_references_give_the_same_bits(K, T, cap):
    """The reference moves in nearly every tile (the last keys come first, and scores grow towards the
    first), so both threads of a row take their scores again, and one's weights go where the other's
    scores are: hundreds of calls have to agree bit by bit."""
    B, Hq, H, S, D = 4, 16, 4, 2048, 128
    q, v = rnd(1, B, Hq, T, D, scale=3.0), rnd(3, B, H, S, D)
    k = (rnd(2, B, H, S, D).float() * torch.linspace(12, 0.01, S, device="cuda")[None, None, :, None]).to(torch.bfloat16)
    qp = i32(np.arange(S - T, S)[None].repeat(B, 0))
    ws = K.attention_chunk_workspace(B, T, Hq, H, D)
    want, lse = C.run(K, q, k, v, qp, None, None, S, cap, ws=ws)
    C.verify(q, k, v, qp, None, None, S, cap, None, want, lse, heads=[0, 7], batches=[0, 3])
    out, wrong = torch.empty_like(want), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        C.run(K, q, k, v, qp, None, None, S, cap, ws=ws, out=out, lse=False)
        wrong += (out.view(torch.int16) != want.view(torch.int16)).sum()
    K.kvc_check_status()
    assert int(wrong) == 0


@pytest.mark.parametrize("T", [20, 200])
@pytest.mark.parametrize("bias", [False, True])
def test_moving_units_give_the_same_bits(K, T, bias):
    """The same over the 8-bit cache, where the scales of both keys and values grow as well."""
    B, Hq, H, D, N = 4, 16, 4, 128, 2048
    so = [h * N for h in range(H + 1)]
    g = torch.exp2(torch.linspace(4, -4, N, device="cuda"))[None, None, :, None]
    k, v = ((rnd(s, B, H, N, D).float() * g).to(torch.bfloat16) for s in (4, 5))
    c = Q.empty_cache(K, B, D, so)
    K.kvc_gather_q8(k, v, torch.arange(N, dtype=torch.int32, device="cuda").repeat(B * H), B, H, N, D, [N] * H, so, *c)
    q, rows, qp = rnd(6, B, Hq, T, D), i32([[N] * H] * B), i32(np.arange(N, N + T)[None].repeat(B, 0))
    sl = Q.slopes_of(Hq, bias)
    ws = K.attention_q8_workspace(B, T, Hq, H, D)
    want, _ = Q.attend(K, q, c, rows, 0, qp, H, so, 0.0, sl, ws=ws)
    out, wrong = torch.empty_like(want), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        Q.attend(K, q, c, rows, 0, qp, H, so, 0.0, sl, ws=ws, out=out, lse=False)
        wrong += (out.view(torch.int16) != want.view(torch.int16)).sum()
    K.kvc_check_status()
    assert torch.isfinite(want).all() and int(wrong) == 0


# ------------------------------------------------------- rows of a tile that are no query
def leave_behind(K, value):
    """Another call of each form leaves full tiles of large queries in shared memory."""
    B, T, Hq, H, D = 8, 256, 32, 8, 128
    q = torch.full((B, Hq, T, D), value, dtype=torch.bfloat16, device="cuda")
    k = rnd(9, B, H, 512, D)
    C.run(K, q, k, k, i32(np.arange(256, 512)[None].repeat(B, 0)), None, None, 512)


@pytest.mark.parametrize("T,G", [(1, 4), (1, 1), (3, 7), (60, 5), (130, 3), (50, 7)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("D", [64, 128])
def test_what_was_in_shared_memory_does_not_matter(K, T, G, cap, D):
    """A tile whose last rows are no query's: what an earlier call left there must not decide when the
    others' reference moves, or which form of the tangent they take."""
    B, H, S = 2, 2, 1500
    Hq = G * H
    q, k, v = rnd(10, B, Hq, T, D), rnd(11, B, H, S, D), rnd(12, B, H, S, D)
    qp = i32(np.arange(S - T, S)[None].repeat(B, 0))
    got = []
    for value in (0.0, 3.0, -40.0, 3e38):
        leave_behind(K, value)
        got.append(C.run(K, q, k, v, qp, None, None, S, cap))
    C.verify(q, k, v, qp, None, None, S, cap, None, *got[0])
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    K.kvc_check_status()


# ------------------------------------------------------- masks
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T", [3, 200])
def test_ranges_at_the_ends_of_their_type(K, T, bias):
    """`last` of -2^31 sees nothing, of 2^31 - 1 all that `first` leaves, `first` of 2^31 - 1 nothing; among
    queries of the same tile that see several tiles of keys."""
    B, Hq, H, S, D = 2, 8, 2, 900, 64
    lo, hi = -(1 << 31), (1 << 31) - 1
    q, k, v = rnd(13, B, Hq, T, D), rnd(14, B, H, S, D), rnd(15, B, H, S, D)
    qp = i32(np.arange(S - T, S)[None].repeat(B, 0))
    first, last = np.zeros((B, T), np.int64), np.full((B, T), S - 1)
    last[:, 0::3] = lo
    last[:, 1::3] = hi
    first[1, :T // 2] = lo
    first[1, T - 1] = hi
    if T > 10:
        first[0, 10], last[0, 10] = hi, lo
        qp[0, 7] = lo                                             # an absent token, whatever its position says
    first, last = i32(first), i32(last)
    sl = C.slopes_of(Hq, bias)
    out, lse = C.run(K, q, k, v, qp, first, last, S, 0.0, sl)
    K.kvc_check_status()
    C.verify(q, k, v, qp, first, last, S, 0.0, sl, out, lse)


def test_queries_before_everything_over_the_cache(K):
    """Positions of -2^31 mark absent tokens too."""
    B, Hq, H, D, T = 2, 8, 2, 64, 40
    n = [300, 200]
    so = K.kvc_q4_layout(H, 1 << 20, n, 0)
    c, _, _ = Q.filled(K, B, H, D, so, n, 16)
    qp = np.arange(800, 800 + T)[None].repeat(B, 0)
    qp[:, ::3] = -(1 << 31)
    qp[1, :] = -(1 << 31)
    qp, rows, q, sl = i32(qp), i32([n] * B), rnd(18, B, Hq, T, D), Q.slopes_of(Hq, True)
    out, lse = Q.attend(K, q, c, rows, 0, qp, H, so, 0.0, sl)
    K.kvc_check_status()
    Q.verify(K, q, c, rows, 0, qp, H, so, 0.0, sl, out, lse)


# ------------------------------------------------------- blocks of values with other scales
def against_own_rows(K, q, c, qp, H, so, out, lse, floor, cap=0.0, slopes=None):
    """Every query against the rows that it sees itself.  A weight times its block's scale (a contribution) is
    off by `floor` of the query's own largest contribution at most, beside the relative roundings of
    attend_util: of row j's output that is floor * max(p s) * |code_j|."""
    B, Hq, T, D = q.shape
    few = Hq // H * T <= 8
    kk, vv = Q.read_all(K, c, B, H, D, so)
    sc = Q.f64(c[2]).reshape(B, -1, 2)[..., 1]
    pos, qpn = c[3].view(B, -1).cpu().numpy(), qp.cpu().numpy()
    qn, on, ln = Q.f64(q), Q.f64(out), Q.f64(lse)
    sl = np.zeros(Hq) if slopes is None else Q.f64(slopes)
    w, qr = (2.0 ** -11, 2.0 ** -24) if few else (2.0 ** -8, 2.0 ** -17)
    for b in range(B):
        for hq in range(Hq):
            h = hq // (Hq // H)
            r = slice(so[h], so[h + 1])
            s = sc[b, so[h] // 16:so[h + 1] // 16].repeat(16)
            k, v, p = kk[b, r], vv[b, r], pos[b, r].astype(np.int64)
            see = (p >= 0) & (p <= qpn[b][:, None])
            far = qpn[b][:, None].astype(np.int64) - p
            ref, rl, mag, x = Q.O.attention_of(qn[b, hq], k, v, see, cap, sl[hq], far)
            some = see.any(1)
            A = float((np.abs(qn[b, hq]) @ np.abs(k).T).max()) / D ** 0.5
            Aq = float(np.abs(qn[b, hq]).max() * np.abs(k).sum(1).max()) / D ** 0.5
            dx = A * 2.0 ** -18 + Aq * qr + 2.0 ** -20 + cap * 2.0 ** -20 + abs(sl[hq]) * float(far.max()) * 2.0 ** -22
            prob = np.where(see, np.exp(x - np.where(some, rl, 0.0)[:, None]), 0.0)
            most = (prob * s).max(1)[:, None]
            codes = see.astype(float) @ (np.abs(v) / s[:, None])
            tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((w + 2 * dx) * mag + floor * most * codes) + 1e-38
            err = np.abs(on[b, hq] - ref)
            assert np.all(err <= tol), (b, hq, float((err / tol).max()))
            assert np.array_equal(np.isneginf(ln[b, hq]), ~some)
            le = np.abs(ln[b, hq][some] - rl[some])
            assert np.all(le <= dx + 2.0 ** -20 * np.abs(rl[some]) + 2.0 ** -20), (b, hq, float(le.max()))


# The tensor cores' form keeps the largest contribution at 2^5 at least, and half a step of its second part is
# 2^-10 (fp16 before it: 2^-17).
MANY_FLOOR = 2.0 ** -15 * (1 + 2.0 ** -7)


@pytest.mark.parametrize("up", [2.0 ** 6, 2.0 ** 9, 2.0 ** 12, 2.0 ** 30])
@pytest.mark.parametrize("T,G", [(9, 1), (40, 4), (5, 4)])
@pytest.mark.parametrize("what", ["unseen", "negligible", "weighty"])
def test_blocks_of_large_values(K, up, T, G, what):
    """Some blocks' values are 2^6 to 2^30 times the others': in rows that come after some of the call's
    queries; with scores that leave them next to no weight; and with weight."""
    blocks_of_large_values(K, up, T, G, what, 2, MANY_FLOOR)


def blocks_of_large_values(K, up, T, G, what, B, floor):
    H, D, N = 2, 64, 1200
    Hq, so = G * H, [0, N, 2 * N]
    q, k, v = rnd(20, B, Hq, T, D, scale=1.5), rnd(21, B, H, N, D), rnd(22, B, H, N, D)
    # of query heads' common direction: what a key has there, a score of 12 / 8 * that
    q[..., 0] = 12.0
    k[..., 0] = 0.0
    big = [(64, 80), (560, 592), (N - 16, N)]
    qp = np.arange(N, N + T)[None].repeat(B, 0)
    for a, e in big if what != "unseen" else big[2:]:
        v[:, :, a:e] = (v[:, :, a:e].float() * up).to(torch.bfloat16)
        if what == "negligible":
            k[:, :, a:e, 0] = -30.0                               # 45 below: e^-45
        elif what == "weighty":
            k[:, :, a:e, 0] = -2.0
    if what == "unseen":
        qp[:, :T // 2] = N - 17 - np.arange(T // 2)               # the first half do not see the last block
    c = Q.empty_cache(K, B, D, so)
    K.kvc_gather_q8(k, v, torch.arange(N, dtype=torch.int32, device="cuda").repeat(2 * B), B, H, N, D, [N, N], so, *c)
    qp = i32(qp)
    out, lse = Q.attend(K, q, c, i32([[N, N]] * B), 0, qp, H, so)
    K.kvc_check_status()
    against_own_rows(K, q, c, qp, H, so, out, lse, floor)


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True)])
@pytest.mark.parametrize("T", [20, 150])
def test_scales_of_values_over_forty_binades(K, order, cap, bias, T):
    """Values that grow and fall by 2^40 over the cache, scores that run against them or with them, a block
    of zeros among them: a reference and a unit that both move, and seldom together."""
    B, Hq, H, D, N = 1, 8, 2, 128, 1600
    so = [0, N, 2 * N]
    g = torch.exp2(torch.linspace(-20, 20, N, device="cuda"))[None, None, :, None]
    q, k = rnd(23, B, Hq, T, D), rnd(24, B, H, N, D)
    v = (rnd(25, B, H, N, D).float() * (g if order == 1 else g.flip(2))).to(torch.bfloat16)
    v[:, :, 800:816] = 0
    q[..., 0] = 4.0
    k[:, 0, :, 0] = torch.linspace(12, -12, N, device="cuda").to(torch.bfloat16)
    k[:, 1, :, 0] = torch.linspace(-40, 40, N, device="cuda").to(torch.bfloat16)
    c = Q.empty_cache(K, B, D, so)
    K.kvc_gather_q8(k, v, torch.arange(N, dtype=torch.int32, device="cuda").repeat(2), B, H, N, D, [N, N], so, *c)
    qp = np.random.default_rng(3).integers(0, N + 50, (B, T))
    qp[0, 3] = -1
    qp, sl = i32(qp), Q.slopes_of(Hq, bias)
    out, lse = Q.attend(K, q, c, i32([[N, N]]), 0, qp, H, so, cap, sl)
    K.kvc_check_status()
    against_own_rows(K, q, c, qp, H, so, out, lse, MANY_FLOOR, cap, sl)


def test_later_tokens_do_not_change_a_query(K):
    """The tokens of a call that come later, with values 2^12 times as large, leave a query's output within
    the bounds of what it sees itself."""
    B, Hq, H, D, N, T = 1, 8, 2, 64, 512, 32
    so = [0, N + T, 2 * (N + T)]
    k, v = rnd(26, B, H, N, D), rnd(27, B, H, N, D)
    nk, nv, q = rnd(28, B, H, T, D), rnd(29, B, H, T, D), rnd(30, B, Hq, T, D)
    qp = i32(np.arange(N, N + T)[None])
    for up in (1.0, 2.0 ** 12):
        nv2 = nv.clone()
        nv2[:, :, 16:] = (nv2[:, :, 16:].float() * up).to(torch.bfloat16)
        c = Q.empty_cache(K, B, D, so)
        idx = torch.arange(N + T, dtype=torch.int32, device="cuda").repeat(2)
        K.kvc_gather_q8(k, v, idx, B, H, N, D, [N, N], so, *c)
        K.kvc_append_q8(nk, nv2, qp, B, H, T, D, so, i32([[N, N]]), *c)
        out, lse = Q.attend(K, q, c, i32([[N, N]]), T, qp, H, so)
        K.kvc_check_status()
        against_own_rows(K, q, c, qp, H, so, out, lse, MANY_FLOOR)


# ------------------------------------------------------- scores of other magnitudes before
@pytest.mark.parametrize("small", [7.0, 100.0, 400.0, -400.0])
@pytest.mark.parametrize("T", [5, 200])
def test_small_scores_behind_far_larger_ones(K, small, T):
    """Sequences with scores around 2^34 in turn with sequences of ordinary ones: a segment's first reference is
    the last one's, whose steps are larger than the scores."""
    B, Hq, H, S, D = 300, 4, 1, 120 if T == 5 else 250, 64
    q, k, v = rnd(31, B, Hq, T, D), rnd(32, B, H, S, D), rnd(33, B, H, S, D)
    q[..., 0] = 2.0 ** 10
    k[..., 0] = small * 8 / 2.0 ** 10
    k[::2, ..., 0] = 2.0 ** 27
    qp = i32(np.arange(S - T, S)[None].repeat(B, 0))
    out, lse = C.run(K, q, k, v, qp, None, None, S)
    K.kvc_check_status()
    C.verify(q, k, v, qp, None, None, S, 0.0, None, out, lse, heads=[0, 3], batches=range(1, B, 26))


@pytest.mark.parametrize("small", [7.0, 100.0, -400.0])
@pytest.mark.parametrize("T", [5, 100])
@pytest.mark.parametrize("level", [2.0 ** 20, 2.0 ** 27])
def test_small_scores_behind_far_larger_ones_over_the_cache(K, small, T, level):
    B, Hq, H, D, N = 300, 4, 1, 64, 112
    so = [0, N]
    q, k, v = rnd(34, B, Hq, T, D), rnd(35, B, H, N, D), rnd(36, B, H, N, D)
    q[..., 0] = 64.0
    k[..., 0] = small * 8 / 64.0
    k[::2, ..., 0] = level * 8 / 64.0
    c = Q.empty_cache(K, B, D, so)
    K.kvc_gather_q8(k, v, torch.arange(N, dtype=torch.int32, device="cuda").repeat(B), B, H, N, D, [N], so, *c)
    qp = i32(np.arange(N, N + T)[None].repeat(B, 0))
    out, lse = Q.attend(K, q, c, i32([[N]] * B), 0, qp, H, so)
    K.kvc_check_status()
    assert torch.isfinite(out).all()
    for b in range(1, B, 26):
        sub = tuple(t.view(B, -1, *t.shape[1:])[b].contiguous() for t in c)
        against_own_rows(K, q[b:b + 1], sub, qp[b:b + 1], H, so, out[b:b + 1], lse[b:b + 1], MANY_FLOOR)


@pytest.mark.parametrize("T", [9, 60])
@pytest.mark.parametrize("level", [2.0 ** 12, 2.0 ** 20, 2.0 ** 27])
def test_large_scores_close_to_one_another(K, T, level):
    """Scores as far up as single steps of fp32 are 2^-11, 2^-3 and 2^4: as good as those steps allow."""
    B, Hq, H, D, N = 2, 4, 2, 128, 700
    so = K.kvc_q4_layout(H, N, [N, N], 0)
    q, k, v = rnd(37, B, Hq, T, D, scale=0.1), rnd(38, B, H, N, D), rnd(39, B, H, N, D)
    q[..., 0] = 16.0
    k[..., 0] = level * 128 ** 0.5 / 16
    # keys of one row in three differ by steps of bf16 in that direction, which decide
    k[:, :, ::3, 0] *= 1 - 2.0 ** -7
    c = Q.empty_cache(K, B, D, so)
    idx = torch.arange(so[1], dtype=torch.int32, device="cuda").clamp(max=N - 1).repeat(2 * B)
    K.kvc_gather_q8(k, v, idx, B, H, N, D, [N, N], so, *c)
    qp = i32(np.arange(N, N + T)[None].repeat(B, 0))
    out, lse = Q.attend(K, q, c, i32([[N, N]] * B), 0, qp, H, so)
    Q.verify(K, q, c, i32([[N, N]] * B), 0, qp, H, so, 0.0, None, out, lse)
    out, lse = C.run(K, q, k, v, qp, None, None, N)
    C.verify(q, k, v, qp, None, None, N, 0.0, None, out, lse)
    K.kvc_check_status()


# ------------------------------------------------------- caches without room
@pytest.mark.parametrize("T", [1, 40])
def test_slots_without_any_row(K, T):
    """A slot table of which no head has a row (budgets of 0 before the first token): zeros, and -inf; counts
    above that are recorded."""
    B, Hq, H, D = 2, 8, 2, 64
    so = [0, 0, 0]
    c = Q.empty_cache(K, 1, D, [0, 16])
    q, qp = rnd(40, B, Hq, T, D), i32(np.arange(T)[None].repeat(B, 0))
    out, lse = Q.attend(K, q, c, i32([[0, 0]] * B), 0, qp, H, so)
    K.kvc_check_status()
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    out, lse = Q.attend(K, q, c, i32([[0, 3]] * B), 0, qp, H, so)
    with pytest.raises(K.KvcError) as e:
        K.kvc_check_status()
    assert e.value.code == K.KVC_ERR_DEVICE
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


# The form for up to 8 query rows: the largest contribution 2^4 units at least, half of fp16's last step.
FEW_FLOOR = 2.0 ** -29


@pytest.mark.parametrize("up", [2.0 ** 9, 2.0 ** 16, 2.0 ** 22, 2.0 ** 40])
@pytest.mark.parametrize("T,G", [(2, 4), (1, 8), (8, 1)])
@pytest.mark.parametrize("what", ["unseen", "negligible", "weighty"])
@pytest.mark.parametrize("B", [2, 24])                             # clusters of CTAs, ranges
def test_blocks_of_large_values_few_rows(K, up, T, G, what, B):
    """The same with up to 8 query rows."""
    if what == "unseen" and T == 1:
        pytest.skip("one token")
    blocks_of_large_values(K, up, T, G, what, B, FEW_FLOOR)


@pytest.mark.parametrize("T", [1, 2, 5, 60])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_queries_over_the_cache(K, T, cap, value):
    """A query row that is not finite gives NaN whatever the form, where it sees a row, and leaves the others'."""
    B, Hq, H, D = 2, 8, 2, 64
    n = [300, 200]
    so = K.kvc_q4_layout(H, 1 << 20, n, 0)
    c, _, _ = Q.filled(K, B, H, D, so, n, 50)
    q, rows = rnd(52, B, Hq, T, D), i32([n, [300, 0]])
    qp = np.full((B, T), 5000)
    qp[0, 0] = 0 if T > 1 else 5000                               # sees the first row alone
    qp = i32(qp)
    bad = q.clone()
    bad[:, 2::4, T - 1, 5] = value
    out, lse = Q.attend(K, bad, c, rows, 0, qp, H, so, cap)
    K.kvc_check_status()
    assert torch.isnan(out[:, 2, T - 1]).all() and torch.isnan(out[0, 6, T - 1]).all()
    assert torch.isnan(lse[:, 2, T - 1]).all()
    assert torch.all(out[1, 6, T - 1] == 0) and torch.isneginf(lse[1, 6, T - 1])      # no rows
    good = torch.ones((B, Hq, T), dtype=torch.bool, device="cuda")
    good[:, 2::4, T - 1] = False
    want, want_lse = Q.attend(K, q, c, rows, 0, qp, H, so, cap)
    out[~good], lse[~good] = want[~good], want_lse[~good]
    Q.verify(K, q, c, rows, 0, qp, H, so, cap, None, out, lse)
