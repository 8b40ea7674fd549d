"""Refusals of the 8-bit cache's entry points and of the chunk attention: every bad
argument is an error before anything is launched (no GPU; the pointers are never
touched).  And the fp64 definition of the 8-bit rows against a plain enumeration."""

import math

import numpy as np
import pytest

from oracle import serve as O


@pytest.fixture(scope="module")
def K():
    from attention_score_kv_gb300 import build
    build.build()
    import attention_score_kv_gb300.kvc as kvc
    return kvc


SLOT = [0, 16, 64]
CACHE = dict(k8=0x4000, v8=0x4400, scale=0x4800)
GATHER = dict(k=0x1000, v=0x2000, idx=0x3000, B=1, H_kv=2, S=100, D=64, K_l=[16, 48], slot_off=SLOT, **CACHE,
              pos=0x5000, stream=0)
APPEND = dict(k=0x1000, v=0x2000, pos_new=0x3000, B=1, H_kv=2, T=3, D=64, slot_off=SLOT, rows=0x3100, **CACHE,
              pos=0x5000, stream=0)
READ = dict(**CACHE, B=1, H_kv=2, D=64, slot_off=SLOT, first=None, n_rows=[16, 48], k_out=0x1000, v_out=0x2000,
            stream=0)
ATTEND = dict(q=0x1000, **CACHE, pos=0x5000, rows=0x3100, extra=1, q_pos=0x6000, B=1, T=1, H_q=4, H_kv=2, D=64,
              slot_off=SLOT, cap=0.0, slopes=None, out=0x7000, lse=0x8000, ws=0x10000, ws_bytes=1 << 40, stream=0)
CHUNK = dict(q=0x1000, k=0x2000, v=0x3000, q_pos=0x4000, first=0x5000, last=0x6000, B=1, T=3, H_q=4, H_kv=2, S=10, D=64,
             cap=0.0, slopes=0x6100, out=0x7000, lse=0x8000, ws=0x10000, ws_bytes=1 << 40, stream=0)
SLOTS = [
    (dict(slot_off=[0, 16, 60]), -1), (dict(slot_off=[-16, 16, 64]), -1), (dict(slot_off=[0, 64, 48]), -1),
    (dict(slot_off=[0, 16, 16 + (1 << 31)]), -2), (dict(slot_off=None), -1),
    (dict(B=0), -1), (dict(H_kv=0), -1), (dict(D=80), -2), (dict(H_kv=129, slot_off=[0] * 130), -2),
    (dict(k8=None), -1), (dict(k8=0x4008), -1), (dict(v8=None), -1), (dict(v8=0x4404), -1), (dict(scale=None), -1),
    (dict(scale=0x4804), -1),
]
MODS = [(dict(cap=c), -1) for c in (-1.0, 2.0 ** -21, 2.0 ** 21, math.inf, math.nan)] + [(dict(slopes=0x6102), -1)]


def refuses(f, args, code):
    f_error = None
    try:
        f(**args)
    except Exception as e:
        f_error = e
    assert getattr(f_error, "code", None) == code, (f_error, code)


@pytest.mark.parametrize("over,code", SLOTS + [
    (dict(K_l=[17, 48]), -1), (dict(K_l=[16, 49]), -1), (dict(K_l=[-1, 4]), -1), (dict(K_l=None), -1),
    (dict(S=0), -1), (dict(S=(1 << 30) + 1), -2), (dict(idx=None), -1), (dict(v=0x2002), -1), (dict(pos=None), -1),
])
def test_gather_refuses(K, over, code):
    if over.get("H_kv") == 129:
        over = {**over, "K_l": [0] * 129}
    refuses(K.kvc_gather_q8, {**GATHER, **over}, code)


@pytest.mark.parametrize("over,code", SLOTS + [
    (dict(T=0), -1), (dict(T=(1 << 30) + 1), -2), (dict(B=1 << 20, T=1 << 20), -2), (dict(rows=None), -1),
    (dict(pos_new=None), -1), (dict(k=None), -1), (dict(pos=0x5002), -1),
])
def test_append_refuses(K, over, code):
    refuses(K.kvc_append_q8, {**APPEND, **over}, code)


@pytest.mark.parametrize("over,code", SLOTS + [
    (dict(n_rows=[17, 48]), -1), (dict(n_rows=[-1, 48]), -1), (dict(n_rows=None), -1),
    (dict(out_off=[0, 8, 64]), -1), (dict(k_out=None), -1), (dict(v_out=0x2004), -1), (dict(first=0x3002), -1),
])
def test_read_refuses(K, over, code):
    if over.get("H_kv") == 129:
        over = {**over, "n_rows": [0] * 129}
    refuses(K.kvc_read_q8, {**READ, **over}, code)


@pytest.mark.parametrize("over,code", SLOTS + MODS + [
    (dict(T=0), -1), (dict(H_q=0), -1), (dict(H_q=5), -1), (dict(extra=-1), -1), (dict(T=1 << 20), -2),
    (dict(H_q=258), -2),                       # 129 query heads a KV head
    (dict(q=None), -1), (dict(q_pos=None), -1), (dict(out=0x7008), -1), (dict(lse=0x8002), -1), (dict(rows=None), -1),
    (dict(pos=None), -1),
])
def test_attention_refuses(K, over, code):
    if over.get("H_kv") == 129:
        over = {**over, "H_q": 129}
    refuses(K.kvc_attention_q8, {**ATTEND, **over}, code)


@pytest.mark.parametrize("over,code", MODS + [
    (dict(B=0), -1), (dict(T=0), -1), (dict(H_q=0), -1), (dict(H_kv=0), -1), (dict(S=0), -1), (dict(H_q=5), -1),
    (dict(D=96), -2), (dict(H_q=258), -2), (dict(S=(1 << 30) + 1), -2), (dict(T=1 << 20), -2), (dict(H_kv=129, H_q=129), -2),
    (dict(q=None), -1), (dict(k=0x2008), -1), (dict(v=None), -1), (dict(q_pos=None), -1), (dict(first=0x5002), -1),
    (dict(last=0x6001), -1), (dict(out=None), -1), (dict(lse=0x8002), -1),
])
def test_chunk_refuses(K, over, code):
    refuses(K.kvc_attention_chunk, {**CHUNK, **over}, code)


def test_workspaces_refuse(K):
    for f in (K.kvc_attention_q8_workspace_size, K.kvc_attention_chunk_workspace_size):
        for args in ((0, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 1, 5, 2, 64), (1, 1, 4, 2, 72), (1, 1, 258, 2, 64)):
            with pytest.raises(K.KvcError):
                f(*args)


def test_compress_refuses(K):
    a = dict(N=1, layer=0, B=1, S=512, C=512, H_q=4, H_kv=2, D=64, W=16, K_l=[128, 128], sink=4, recent=16, pool_k=1,
             b_s=128, q_win=0x1000, k=0x2000, v=0x3000, slot_off=[0, 128, 256], **CACHE, pos=0x6000, ws=0x10000,
             ws_bytes=1 << 30, stream=0)
    for over, code in [(dict(slot_off=[0, 112, 256]), -1), (dict(slot_off=[0, 130, 260]), -1), (dict(k8=None), -1),
                       (dict(scale=0x4804), -1), (dict(pos=None), -1), (dict(H_kv=0), -1), (dict(layer=1), -1),
                       (dict(K_l=[19, 128]), -1), (dict(v=None), -1)]:
        refuses(K.kvc_compress_layer_q8, {**a, **over}, code)


def test_tensors_are_looked_at(K):
    import torch
    for f, args, name, bad in (
            (K.kvc_gather_q8, GATHER, "k8", torch.zeros(64 * 64, dtype=torch.int8)),
            (K.kvc_append_q8, APPEND, "scale", torch.zeros(8, dtype=torch.float64)),
            (K.kvc_read_q8, READ, "v8", torch.zeros(64 * 64 - 1, dtype=torch.uint8)),
            (K.kvc_attention_q8, ATTEND, "slopes", torch.zeros(3)),
            (K.kvc_attention_q8, ATTEND, "ws", torch.zeros(512, dtype=torch.uint8)),
            (K.kvc_attention_chunk, CHUNK, "first", torch.zeros(3, dtype=torch.int64)),
            (K.kvc_attention_chunk, CHUNK, "q", torch.zeros((1, 4, 3, 128), dtype=torch.bfloat16)[..., ::2])):
        with pytest.raises(K.KvcError) as ei:
            f(**{**args, name: bad})
        assert ei.value.code == K.KVC_ERR_INVALID_ARG and name in str(ei.value)


# ------------------------------------------------------------------ the definition
def test_scales_are_the_least_that_hold():
    for top in [448.0, 448.0 * 2 ** -20, 449.0, 447.0, 1e-40, 0.0, 3.3e38, 1.0] + list(np.random.default_rng(0).lognormal(0, 20, 200)):
        s = float(O.scale8(top))
        assert math.log2(s) == round(math.log2(s)) and top <= 448 * s
        assert s == 2.0 ** -100 or top > 448 * (s / 2)


def test_rows_are_the_nearest_values():
    """Against every e4m3 value of a block's scale, by distance."""
    g = np.random.default_rng(1)
    x = g.normal(size=(40, 64)) * 2.0 ** g.integers(-12, 12, (40, 1))
    got, s = O.held8(x)
    grid = np.concatenate((O.E4M3, -O.E4M3))
    for i in range(40):
        near = np.abs(x[i][:, None] - grid * s[i // 16]).min(1)
        assert np.array_equal(np.abs(got[i] - x[i]), near)


def test_an_append_holds_what_a_block_written_at_once_does():
    """New rows that need no larger scale leave the block as a gather of all would, and a larger
    one rounds the earlier rows anew: the same but for e4m3's subnormals."""
    g = np.random.default_rng(2)
    x = g.normal(size=(37, 64))
    x[5] *= 8
    held, s = O.held8(x[:20])
    got, gs = O.append8(held, s, x[20:])
    want, ws = O.held8(x)
    assert np.array_equal(got, want) and np.array_equal(gs, ws)
    x[22] *= 2.0 ** 5
    got, gs = O.append8(held, s, x[20:])
    want, ws = O.held8(x)
    assert np.array_equal(gs, ws) and np.all(np.abs(got - want) <= ws[1] * 2.0 ** -9)
