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
