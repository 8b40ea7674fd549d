"""Refusals of the serving entry points: every bad argument is an error before
anything is launched (no GPU; the pointers are never touched)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def K():
    from attention_score_kv_gb300 import build
    build.build()
    import attention_score_kv_gb300.kvc as kvc
    return kvc


ROPE = dict(q=0x1000, k=0x2000, v=0x3000, B=2, T=3, H_q=4, H_kv=2, D=64, q_ld=512, k_ld=512, v_ld=512, R=64,
            interleaved=0, q_weight=0x4000, k_weight=0x5000, eps=1e-6, inv_freq=0x6000, pos=0x7000, S=8, row0=5,
            q_out=0x8000, k_act=0x9000, v_act=0xa000, stream=0)


@pytest.mark.parametrize("over,code", [
    (dict(B=0), -1), (dict(T=0), -1), (dict(H_q=0), -1), (dict(H_kv=0), -1),
    (dict(D=96), -2), (dict(R=24), -1), (dict(R=80), -1), (dict(R=-16), -1),
    (dict(interleaved=2), -1),
    (dict(row0=-1), -1), (dict(row0=6), -1), (dict(S=2, row0=0), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(q_ld=248), -1), (dict(q_ld=260), -1), (dict(k_ld=120), -1), (dict(v_ld=132), -1),
    (dict(q=None), -1), (dict(k=0x2008), -1), (dict(v=None), -1), (dict(v_act=None), -1),
    (dict(q_weight=0x4002), -1), (dict(inv_freq=None), -1), (dict(pos=None), -1), (dict(k_act=None), -1),
    (dict(B=1 << 20, T=1 << 12, S=1 << 13), -2), (dict(H_q=70000, q_ld=1 << 23), -2),
])
def test_norm_rope_refuses(K, over, code):
    with pytest.raises(K.KvcError) as ei:
        K.kvc_qk_norm_rope(**{**ROPE, **over})
    assert ei.value.code == code


SLOT = [0, 16, 64]
GATHER = dict(k=0x1000, v=0x2000, idx=0x3000, B=1, H_kv=2, S=100, D=64, K_l=[16, 48], slot_off=SLOT, cache=0x4000,
              pos=0x5000, stream=0)
APPEND = dict(k=0x1000, v=0x2000, pos_new=0x3000, B=1, H_kv=2, T=3, D=64, slot_off=SLOT, rows=0x3100, cache=0x4000,
              pos=0x5000, stream=0)
READ = dict(cache=0x4000, B=1, H_kv=2, D=64, slot_off=SLOT, first=None, n_rows=[16, 48], k_out=0x1000, v_out=0x2000,
            stream=0)
ATTEND = dict(q=0x1000, cache=0x4000, pos=0x5000, rows=0x3100, extra=1, q_pos=0x6000, B=1, T=1, H_q=4, H_kv=2, D=64,
              slot_off=SLOT, out=0x7000, lse=0x8000, ws=0x10000, ws_bytes=1 << 40, stream=0)
SLOTS = [
    (dict(slot_off=[0, 16, 60]), -1),          # not a multiple of 16
    (dict(slot_off=[-16, 16, 64]), -1),
    (dict(slot_off=[0, 64, 48]), -1),          # out of order
    (dict(slot_off=[0, 16, 16 + (1 << 31)]), -2),
    (dict(slot_off=None), -1),
    (dict(B=0), -1), (dict(H_kv=0), -1), (dict(D=80), -2), (dict(H_kv=129, slot_off=[0] * 130), -2),
    (dict(cache=None), -1), (dict(cache=0x4008), -1),
]


@pytest.mark.parametrize("over,code", SLOTS + [
    (dict(K_l=[17, 48]), -1),                  # slot 0 has 16 rows
    (dict(K_l=[16, 49]), -1), (dict(K_l=[-1, 4]), -1), (dict(K_l=None), -1),
    (dict(S=0), -1), (dict(S=(1 << 30) + 1), -2), (dict(idx=None), -1), (dict(v=0x2002), -1), (dict(pos=None), -1),
])
def test_gather_refuses(K, over, code):
    if over.get("H_kv") == 129:
        over = {**over, "K_l": [0] * 129}
    with pytest.raises(K.KvcError) as ei:
        K.kvc_gather_q4(**{**GATHER, **over})
    assert ei.value.code == code


@pytest.mark.parametrize("over,code", SLOTS + [
    (dict(T=0), -1), (dict(T=(1 << 30) + 1), -2), (dict(B=1 << 20, T=1 << 20), -2), (dict(rows=None), -1),
    (dict(pos_new=None), -1), (dict(k=None), -1), (dict(pos=0x5002), -1),
])
def test_append_refuses(K, over, code):
    with pytest.raises(K.KvcError) as ei:
        K.kvc_append_q4(**{**APPEND, **over})
    assert ei.value.code == code


@pytest.mark.parametrize("over,code", SLOTS + [
    (dict(n_rows=[17, 48]), -1), (dict(n_rows=[-1, 48]), -1), (dict(n_rows=None), -1),
    (dict(out_off=[0, 8, 64]), -1), (dict(k_out=None), -1), (dict(v_out=0x2004), -1), (dict(first=0x3002), -1),
])
def test_read_refuses(K, over, code):
    if over.get("H_kv") == 129:
        over = {**over, "n_rows": [0] * 129}
    with pytest.raises(K.KvcError) as ei:
        K.kvc_read_q4(**{**READ, **over})
    assert ei.value.code == code


@pytest.mark.parametrize("over,code", SLOTS + [
    (dict(T=0), -1), (dict(H_q=0), -1), (dict(H_q=5), -1), (dict(extra=-1), -1), (dict(T=1 << 20), -2),
    (dict(B=1 << 24, H_kv=1, H_q=256, slot_off=[0, 16]), -2),
    (dict(q=None), -1), (dict(q_pos=None), -1), (dict(out=0x7008), -1), (dict(lse=0x8002), -1), (dict(rows=None), -1),
])
def test_attention_refuses(K, over, code):
    if over.get("H_kv") == 129:
        over = {**over, "H_q": 129}
    with pytest.raises(K.KvcError) as ei:
        K.kvc_attention_q4(**{**ATTEND, **over})
    assert ei.value.code == code


@pytest.mark.parametrize("args", [(0, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 1, 5, 2, 64), (1, 1, 4, 2, 72)])
def test_attention_workspace_refuses(K, args):
    with pytest.raises(K.KvcError):
        K.kvc_attention_q4_workspace_size(*args)


def test_compress_q4_refuses(K):
    a = dict(N=1, layer=0, B=1, S=512, C=512, H_q=4, H_kv=2, D=64, W=16, K_l=[128, 128], sink=4, recent=16, pool_k=1,
             b_s=128, q_win=0x1000, k=0x2000, v=0x3000, slot_off=[0, 128, 256], cache=0x4000, pos=0x6000, ws=0x10000,
             ws_bytes=1 << 30, stream=0)
    for over, code in [(dict(slot_off=[0, 112, 256]), -1), (dict(slot_off=[0, 130, 260]), -1), (dict(cache=None), -1),
                       (dict(H_kv=0), -1), (dict(layer=1), -1), (dict(K_l=[19, 128]), -1), (dict(v=None), -1)]:
        with pytest.raises(K.KvcError) as ei:
            K.kvc_compress_layer_q4(**{**a, **over})
        assert ei.value.code == code, over


def test_slots(K):
    so = K.kvc_q4_layout(4, 100, [0, 1, 90, 500], 7)
    assert list(so) == [0, 16, 32, 144, 256]       # 7, 8, 97 and 107 rows
    assert isinstance(so, ctypes.Array)
    for bad in [(0, 100, [], 0), (1, 0, [4], 0), (1, 10, [-1], 0), (1, 10, [4], -1)]:
        with pytest.raises(K.KvcError) as ei:
            K.kvc_q4_layout(*bad)
        assert ei.value.code == -1


def test_host_tensors_and_wrong_types_are_refused(K):
    import torch
    q = torch.zeros((2, 3, 4 * 64), dtype=torch.bfloat16)
    with pytest.raises(K.KvcError) as ei:          # wrong type, before any look at the device
        K.kvc_qk_norm_rope(**{**ROPE, "q": q.float()})
    assert ei.value.code == -1 and "float32" in str(ei.value)
    with pytest.raises(K.KvcError) as ei:          # no tokens: refused with the tensors as they are
        K.kvc_qk_norm_rope(**{**ROPE, "q": q, "T": 0})
    assert ei.value.code == -1
    with pytest.raises(K.KvcError) as ei:
        K.kvc_read_q4(**{**READ, "slot_off": [0, 16]})   # too short a host array
    assert ei.value.code == -1
    with pytest.raises(K.KvcError) as ei:
        K.kvc_append_q4(**{**APPEND, "pos_new": torch.zeros(2, dtype=torch.int32)})
    assert ei.value.code == -1 and "pos_new" in str(ei.value)


def test_host_arrays_of_every_kind_are_taken(K):
    """Lists, tensors, arrays of the right and of another type: all reach the same check (K_l[1]
    = 49 does not fit its slot)."""
    import array
    import numpy as np
    import torch
    for make in (list, tuple, torch.tensor, lambda x: torch.tensor(x, dtype=torch.int32), np.array,
                 lambda x: np.array(x, dtype=np.int32), lambda x: np.array(x, dtype=np.int64),
                 lambda x: array.array("i", x), lambda x: array.array("q", x), lambda x: (ctypes.c_int32 * 2)(*x), lambda x: (ctypes.c_int64 * 2)(*x)):
        with pytest.raises(K.KvcError) as ei:
            K.kvc_gather_q4(**{**GATHER, "K_l": make([16, 49])})
        assert ei.value.code == -1 and "out_off" in str(ei.value), make
    for make in (list, lambda x: (ctypes.c_int64 * 3)(*x), np.array, torch.tensor):
        with pytest.raises(K.KvcError) as ei:
            K.kvc_gather_q4(**{**GATHER, "slot_off": make([0, 16, 60])})
        assert ei.value.code == -1 and "slot_off" in str(ei.value)
    with pytest.raises(K.KvcError) as ei:                      # every other value of an array
        K.kvc_gather_q4(**{**GATHER, "K_l": np.array([16, 0, 49, 0], dtype=np.int32)[::2]})
    assert ei.value.code == -1 and "out_off" in str(ei.value)


def test_arguments_of_another_type_are_type_errors(K):
    for over in (dict(B="1"), dict(S=1.5), dict(k="x"), dict(K_l=3), dict(stream="s")):
        with pytest.raises((TypeError, AttributeError)):
            K.kvc_gather_q4(**{**GATHER, **over})
    with pytest.raises(OverflowError):
        K.kvc_gather_q4(**{**GATHER, "S": 1 << 40})
    with pytest.raises(TypeError):
        K.kvc_qk_norm_rope(**{**ROPE, "eps": "small"})


def test_refused_calls_leave_no_references(K):
    """Arguments are held no longer than the call, whichever check ends it."""
    import sys

    import torch
    t = torch.zeros((2, 3, 256), dtype=torch.bfloat16)
    slot, kl = (ctypes.c_int64 * 3)(*SLOT), [16, 49]

    def calls():
        for f, a in ((K.kvc_gather_q4, {**GATHER, "slot_off": slot, "K_l": kl}),
                     (K.kvc_gather_q4, {**GATHER, "slot_off": slot, "k": t}),
                     (K.kvc_gather_q4, {**GATHER, "slot_off": slot, "stream": t}),
                     (K.kvc_append_q4, {**APPEND, "slot_off": slot, "k": t}),
                     (K.kvc_read_q4, {**READ, "slot_off": slot, "n_rows": kl}),
                     (K.kvc_attention_q4, {**ATTEND, "slot_off": slot, "q": t, "T": 0}),
                     (K.kvc_qk_norm_rope, {**ROPE, "q": t, "q_ld": 256}),
                     (K.kvc_qk_norm_rope, {**ROPE, "q": t.float()})):
            try:
                f(**a)
            except (K.KvcError, AttributeError):
                pass
            else:
                raise AssertionError("not refused")

    calls()
    seen = (t, slot, kl, torch.bfloat16, K.KvcError, None)
    before = [sys.getrefcount(x) for x in seen]
    for _ in range(50):
        calls()
    after = [sys.getrefcount(x) for x in seen]
    assert all(abs(a - b) < 40 for a, b in zip(after, before)), (before, after)


@pytest.mark.parametrize("value", [2 ** 31, -2 ** 31 - 1, 2 ** 32 + 16])
def test_host_values_that_do_not_fit_are_refused(K, value):
    """A list's values become 32-bit integers: none may wrap around on the way."""
    with pytest.raises(K.KvcError) as e:
        K.kvc_q4_layout(2, 64, [16, value], 0)
    assert e.value.code == K.KVC_ERR_INVALID_ARG and "K_l" in str(e.value)
    with pytest.raises(K.KvcError) as e:
        K.kvc_read_q4(**{**READ, "n_rows": [value] * READ["H_kv"]})
    assert e.value.code == K.KVC_ERR_INVALID_ARG and "n_rows" in str(e.value)
    with pytest.raises(K.KvcError):
        K.kvc_read_q4(**{**READ, "slot_off": [2 ** 64] * (READ["H_kv"] + 1)})


def test_a_workspace_smaller_than_stated_is_refused(K):
    """ws_bytes speaks for a raw pointer; a tensor has to hold what is stated."""
    import torch
    ws = torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(K.KvcError) as ei:
        K.kvc_attention_q4(**{**ATTEND, "ws": ws, "ws_bytes": 1 << 40})
    assert ei.value.code == K.KVC_ERR_INVALID_ARG and "ws holds 512" in str(ei.value)
    with pytest.raises(K.KvcError) as ei:
        K.kvc_compress_layer_q4(1, 0, 1, 512, 512, 4, 2, 64, 16, [128, 128], 4, 16, 1, 128, 0x1000, 0x2000, 0x3000,
                                [0, 128, 256], 0x4000, 0x6000, ws, ws_bytes=1 << 40, stream=0)
    assert ei.value.code == K.KVC_ERR_INVALID_ARG and "ws holds 512" in str(ei.value)


@pytest.mark.parametrize("value", [16.5, -0.25, float("nan"), float("inf")])
def test_host_values_that_are_no_integers_are_refused(K, value):
    """Row counts are not rounded on the way; whole numbers of another type are taken."""
    import numpy as np
    import torch
    for make in (list, np.array, torch.tensor, lambda x: [np.float32(y) for y in x]):
        with pytest.raises(K.KvcError) as e:
            K.kvc_q4_layout(2, 64, make([16.0, value]), 0)
        assert e.value.code == K.KVC_ERR_INVALID_ARG and "K_l" in str(e.value)
        with pytest.raises(K.KvcError) as e:
            K.kvc_read_q4(**{**READ, "n_rows": make([16.0, value])})
        assert e.value.code == K.KVC_ERR_INVALID_ARG and "n_rows" in str(e.value)
        with pytest.raises(K.KvcError) as e:
            K.kvc_gather_q4(**{**GATHER, "slot_off": make([0.0, 16.0, value])})
        assert e.value.code == K.KVC_ERR_INVALID_ARG and "slot_off" in str(e.value)
        assert list(K.kvc_q4_layout(2, 64, make([16.0, 17.0]), 0)) == [0, 16, 48]


def test_the_compress_needs_no_marshalling_module(K):
    """Without the module of csrc/kvc_python.c (another Python, no headers) the library's other calls
    work, and a decoding step's calls say what is missing."""
    import os
    import subprocess
    import sys
    code = """if True:
        import sys
        sys.modules["attention_score_kv_gb300._binding"] = None
        import attention_score_kv_gb300.kvc as K
        assert K.kvc_retained_layout(2, 100, [5, 7]) == [0, 5, 12]
        assert list(K.kvc_q4_layout(2, 100, [5, 17], 0)) == [0, 16, 48]
        try:
            K.kvc_gather(*[0x1000] * 3, 0, 2, 100, 64, [5, 7], *[0x1000] * 3, stream=0)
            raise AssertionError("not refused")
        except K.KvcError as e:
            assert e.code == K.KVC_ERR_INVALID_ARG
        try:
            K.kvc_append_q4(*[0x1000] * 3, 1, 1, 1, 64, [0, 16], *[0x1000] * 3, stream=0)
            raise AssertionError("not refused")
        except ImportError as e:
            assert "attention_score_kv_gb300.build" in str(e)
        print("fine")
    """
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert p.returncode == 0 and "fine" in p.stdout, p.stderr


def test_the_library_is_built_without_pythons_headers(K, tmp_path, monkeypatch):
    import sysconfig

    from attention_score_kv_gb300 import build
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(sysconfig, "get_path", lambda name: str(tmp_path))
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build() == build.LIB
    assert not (tmp_path / "_binding.so").exists()
