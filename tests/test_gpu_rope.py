"""kvc_qk_norm_rope against the fp64 definition.

Tolerance: the result is rounded once to bf16, at most 2^-8 of its value.  The
fp32 steps before it: the sum of D <= 128 squares and rsqrt (relative error
below 2^-18 together), two products, the angle's sine and cosine (absolute
error below 2^-21) and the rotation's two products and sum; with h the length
of the rotated pair that is below 2^-17 h, and it can move the rounding by as
much again.
"""

import numpy as np
import pytest
import torch

from oracle import serve as O

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


def check_heads(got, x, w, eps, inv_freq, pos, R, inter):
    """got, x [B, H, T, D]; pos [B, T]."""
    for b in range(x.shape[0]):
        for h in range(x.shape[1]):
            ref = O.norm_rope(x[b, h], w, eps, inv_freq, pos[b], R, inter)
            plain = O.norm_rope(x[b, h], w, eps, None, pos[b], 0, inter)
            size = np.abs(plain)
            if R:
                i = np.arange(R // 2)
                p, q = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
                size[:, p] = size[:, q] = np.hypot(plain[:, p], plain[:, q])
            err = np.abs(got[b, h] - ref)
            assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * size), (b, h, err.max())


CASES = [
    # B, T, Hq, Hkv, D, R, inter, norm, S, row0, first position
    (1, 1, 32, 8, 128, 128, False, True, 1, 0, 65536),
    (3, 1, 5, 1, 128, 128, False, False, 4, 2, 0),
    (2, 7, 4, 2, 64, 64, True, True, 9, 1, 131071),
    (1, 33, 3, 3, 64, 32, False, True, 40, 7, 12345678),
    (2, 5, 7, 1, 128, 16, True, True, 5, 0, 2147483000),
    (1, 300, 6, 2, 128, 64, False, False, 1000, 700, 7),
    (5, 2, 2, 1, 64, 0, False, True, 2, 0, 3),
    (67, 3, 8, 2, 128, 128, True, True, 3, 0, 99999),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("fused", [True, False])
def test_norm_rope(K, case, fused):
    B, T, Hq, H, D, R, inter, norm, S, row0, p0 = case
    g = torch.Generator().manual_seed(B * 1000 + T)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    if fused:      # one projection's output, with room behind each token
        ld = (Hq + 2 * H) * D + 24
        x = rnd(B, T, ld)
        q, k, v = x[..., :Hq * D], x[..., Hq * D:(Hq + H) * D], x[..., (Hq + H) * D:(Hq + 2 * H) * D]
        lds = (ld, ld, ld)
    else:
        q, k, v = rnd(B, T, Hq, D), rnd(B, T, H, D), rnd(B, T, H, D)
        lds = (Hq * D, H * D, H * D)
    qw, kw = (rnd(D) + 1, rnd(D) * 0.5 + 1) if norm else (None, None)
    inv = (1e4 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))).float().cuda()
    pos = (p0 + 3 * torch.arange(B)[:, None] + torch.arange(T)).to(torch.int32).cuda()
    q_out = torch.full((B, Hq, T, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    k_act, v_act = rnd(B, H, S, D), rnd(B, H, S, D)
    k0, v0 = k_act.clone(), v_act.clone()
    eps = 1e-6
    K.kvc_qk_norm_rope(q, k, v, B, T, Hq, H, D, *lds, R, int(inter), qw, kw, eps, inv, pos, S, row0, q_out, k_act,
                       v_act)
    K.kvc_check_status()
    heads = lambda t, n: f64(t.reshape(B, T, n, D).transpose(1, 2))
    wq, wk = (f64(qw), f64(kw)) if norm else (None, None)
    check_heads(f64(q_out), heads(q, Hq), wq, eps, f64(inv), pos.cpu().numpy(), R, inter)
    check_heads(f64(k_act[:, :, row0:row0 + T]), heads(k, H), wk, eps, f64(inv), pos.cpu().numpy(), R, inter)
    assert torch.equal(v_act[:, :, row0:row0 + T], v.reshape(B, T, H, D).transpose(1, 2))
    for new, old in ((k_act, k0), (v_act, v0)):        # every other position is as it was
        assert torch.equal(new[:, :, :row0], old[:, :, :row0])
        assert torch.equal(new[:, :, row0 + T:], old[:, :, row0 + T:])


def test_negative_positions_turn_the_other_way(K):
    D, inv = 64, torch.tensor([0.7 ** i for i in range(32)], device="cuda")
    x = torch.randn((1, 1, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for p in (-1, -100000, -2 ** 31, 2 ** 31 - 1):
        q, k = (torch.empty((1, 1, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pos = torch.tensor([[p]], dtype=torch.int32, device="cuda")
        K.kvc_qk_norm_rope(x, x, None, 1, 1, 1, 1, D, D, D, D, D, 0, None, None, 0.0, inv, pos, 1, 0, q, k, None)
        check_heads(f64(q), f64(x)[:, :, None], None, 0.0, f64(inv), np.array([[p]]), D, False)
        assert torch.equal(q, k)


def test_extreme_values(K):
    """A zero head stays zero, NaN and infinity stay in their own head."""
    D = 128
    x = torch.randn((1, 1, 4 * D), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    x[..., :D] = 0
    x[..., D + 5] = float("inf")
    x[..., 2 * D + 1] = float("nan")
    x = x.cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    q = torch.empty((1, 4, 1, D), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((1, 1, 1, D), dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([[11]], dtype=torch.int32, device="cuda")
    inv = torch.full((D // 2,), 0.1, device="cuda")
    K.kvc_qk_norm_rope(x, x[..., :D], None, 1, 1, 4, 1, D, 4 * D, 4 * D, D, D, 0, w, w, 1e-6, inv, pos, 1, 0, q, k,
                       None)
    assert torch.all(q[0, 0] == 0) and torch.isnan(q[0, 2]).all() and torch.isfinite(q[0, 3]).all()
    assert torch.isnan(q[0, 1, 0, 5]) and torch.all(k == 0)


def test_wrong_strides_are_refused(K):
    x = torch.zeros((2, 3, 512), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros((2, 4, 3, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    inv = torch.zeros(32, device="cuda")
    call = lambda q, ld, out=o: K.kvc_qk_norm_rope(q, x[..., 256:384], None, 2, 3, 4, 2, 64, ld, 512, 512, 64, 0, None,
                                                   None, 0.0, inv, pos, 3, 0, out, o, None)
    for bad in (lambda: call(x[..., :256], 256), lambda: call(x[:, :, 0:512:2], 512),
                lambda: call(x.transpose(0, 1)[..., :256], 512), lambda: call(x[..., :256], 512, o[:1])):
        with pytest.raises(K.KvcError):
            bad()
