"""Cases of the serving operators around the retained cache: the norm and
rotation of queries and keys, the 4-bit retained cache (gather into it, append
to it, read it back) and attention over it.

``own`` False computes the plain forms with elementary torch operations;
``own`` True makes the calls of ``attention_score_kv_gb300.kvc``.

The 4-bit cache stores blocks of 16 rows.  A row is held as e2m1 codes with one
e4m3 scale per 16 values; ``unpack`` below spells the block's bytes out.
"""

import ctypes
import math

import torch

own = False

EPS = 1e-6
THETA = 1e6            # rotation base
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One decoding step of one request: latency only (Llama-3.1-8B heads).
        dict(name="rotate one token", op="rotate", B=1, T=1, H_q=32, H_kv=8, D=128, R=128, inter=False, norm=True,
             S=1, row0=0, pos0=65536),
        # A decoding step of a batch, no norm weights (Qwen2.5-14B heads).
        dict(name="rotate 96 requests", op="rotate", B=96, T=1, H_q=40, H_kv=8, D=128, R=128, inter=False,
             norm=False, S=1, row0=0, pos0=32768),
        # A prefill chunk of the layer-major schedule into the active layer's buffers.
        dict(name="rotate a chunk of 2048", op="rotate", B=1, T=2048, H_q=32, H_kv=8, D=128, R=128, inter=False,
             norm=True, S=8192, row0=4096, pos0=4096),
        # A ragged last chunk, head dim 64, half of it rotated, pairs side by side.
        dict(name="rotate a ragged chunk", op="rotate", B=3, T=1537, H_q=4, H_kv=2, D=64, R=32, inter=True,
             norm=True, S=2048, row0=511, pos0=131071),
        # The retained rows of a Llama-3.1-8B layer at 8K, 1024 per head.
        dict(name="gather 1024 of 8K", op="gather", B=1, H_kv=8, S=8192, D=128, keep=1024, uneven=False),
        # Unequal per-head budgets, 30% of 32K on average, batch 4 (Qwen2.5-14B layer).
        dict(name="gather uneven of 32K", op="gather", B=4, H_kv=8, S=32768, D=128, keep=9830, uneven=True),
        # The new token of one request joins the cache.
        dict(name="append one token", op="append", B=1, H_kv=8, T=1, D=128, keep=4096, uneven=False),
        # Five draft tokens of a batch, every sequence at a row of its own.
        dict(name="append 5 tokens of 64", op="append", B=64, H_kv=8, T=5, D=128, keep=1031, uneven=False),
        # One token over TideKV's main budget of 4096 rows per head.
        dict(name="attend one token, 4096 rows", op="attend", B=1, T=1, H_q=32, H_kv=8, D=128, keep=4096,
             uneven=False),
        # One token of four requests over unequal budgets (Qwen2.5-14B layer).
        dict(name="attend one token, uneven", op="attend", B=4, T=1, H_q=40, H_kv=8, D=128, keep=9830, uneven=True),
        # A full serving batch, one token each (Mistral-7B heads, budget 4096).
        dict(name="attend 64 requests", op="attend", B=64, T=1, H_q=32, H_kv=8, D=128, keep=4096, uneven=False),
        # The prompt of a follow-up turn: 512 new tokens over the retained rows and themselves.
        dict(name="attend a turn of 512", op="attend", B=1, T=512, H_q=32, H_kv=8, D=128, keep=4096, uneven=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "gather", "append", "attend", "attend"))
    D = rng.choice((64, 128, 128))
    H_kv = rng.choice((1, 2, 4, 8, 8))
    G = rng.choice((1, 2, 4, 5, 7, 8))
    if op == "rotate":
        T = _log(rng, 1, 2048)
        B = max(1, min(_log(rng, 1, 96), 12000 // (T * (G + 2))))
        R = rng.choice((D, D, D // 2))
        S = T + rng.randrange(0, 1000)
        return dict(op=op, B=B, T=T, H_q=H_kv * G, H_kv=H_kv, D=D, R=R, inter=rng.random() < 0.3,
                    norm=rng.random() < 0.6, S=S, row0=rng.randrange(0, S - T + 1), pos0=_log(rng, 1, 400000))
    if op == "gather":
        S = _log(rng, 128, 65536)
        keep = min(S, _log(rng, 16, 9830))
        B = max(1, min(_log(rng, 1, 8), 39320 // keep, 131072 // S))
        return dict(op=op, B=B, H_kv=H_kv, S=S, D=D, keep=keep, uneven=rng.random() < 0.5)
    keep = _log(rng, 16, 16384)
    if op == "append":
        B = max(1, min(_log(rng, 1, 64), 262144 // keep))
        return dict(op=op, B=B, H_kv=H_kv, T=rng.choice((1, 1, 2, 3, 5, 8, 17, 33)), D=D, keep=keep,
                    uneven=rng.random() < 0.3)
    T = rng.choice((1, 1, 1, 2, 3, 5, 8, _log(rng, 9, 512)))
    B = max(1, min(_log(rng, 1, 64), 262144 // keep, 2 * 10 ** 6 // (T * G * keep)))
    return dict(op=op, B=B, T=T, H_q=H_kv * G, H_kv=H_kv, D=D, keep=keep, uneven=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs
def _kept(c):
    """Retained rows of each KV head: equal, or spread 1:3 around the mean."""
    H, keep = c["H_kv"], c["keep"]
    if not c["uneven"] or H == 1:
        return [keep] * H
    w = [1.0 / (0.25 + 0.5 * ((h * 5) % H) / (H - 1)) for h in range(H)]
    most = c.get("S", 1 << 30)
    return [max(1, min(most, int(keep * H * x / sum(w)))) for x in w]


def _slots(kept, extra):
    """First row of each head's slot (multiples of 16) and, last, a batch element's rows."""
    off = [0]
    for n in kept:
        off.append(off[-1] + (n + extra + 15) // 16 * 16)
    return off


def _rows_of(kept, S, gen):
    """Ascending positions of `kept` rows out of S, one row of the result."""
    return torch.sort(torch.randperm(S, generator=gen, device="cuda")[:kept]).values.to(torch.int32)


def _randn(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


def _cache(c, gen, extra):
    """A cache as earlier gathers and appends left it: codes and scales of normal
    values, positions, and how many rows each sequence's heads hold."""
    B, H, D = c["B"], c["H_kv"], c["D"]
    kept = _kept(c)
    room = 1 + max(kept) // 8
    off = _slots(kept, extra + room)
    R = off[-1]
    cache = torch.empty((B, R // 16, 18 * D), dtype=torch.uint8, device="cuda")
    for b0 in range(0, B, 8):
        n = min(8, B - b0)
        cache[b0:b0 + n] = pack(*(quantise(_randn(gen, n, R, D)) for _ in range(2)))
    S0 = 4 * max(kept)
    age = torch.randint(0, room, (B,), generator=gen, device="cuda", dtype=torch.int32)   # tokens decoded so far
    pos = torch.full((B, R), -1, dtype=torch.int32, device="cuda")
    for h, n in enumerate(kept):
        r = torch.arange(off[h + 1] - off[h] - n, device="cuda", dtype=torch.int32)
        pos[:, off[h]:off[h] + n] = _rows_of(n, S0, gen)
        pos[:, off[h] + n:off[h + 1]] = S0 + r
    rows = torch.tensor(kept, dtype=torch.int32, device="cuda")[None, :] + age[:, None]
    return kept, off, cache, pos, rows, age, S0


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = dict(c=c)
    D, B = c["D"], c["B"]
    if c["op"] == "rotate":
        T, Hq, H, R, S = c["T"], c["H_q"], c["H_kv"], c["R"], c["S"]
        # the projection's output: queries, keys and values of a token side by side
        st["qkv"] = _randn(gen, B, T, (Hq + 2 * H) * D)
        st["qw"] = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16) if c["norm"] else None
        st["kw"] = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16) if c["norm"] else None
        st["inv_freq"] = (THETA ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda()
        start = c["pos0"] + torch.randint(0, 64, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        st["pos"] = start + torch.arange(T, device="cuda", dtype=torch.int32)
        st["q_out"] = torch.empty((B, Hq, T, D), dtype=torch.bfloat16, device="cuda")
        st["k_act"] = _randn(gen, B, H, S, D)
        st["v_act"] = _randn(gen, B, H, S, D)
        return st
    H = c["H_kv"]
    if c["op"] == "gather":
        S = c["S"]
        kept = _kept(c)
        off = _slots(kept, 64)
        st["k"], st["v"] = _randn(gen, B, H, S, D, scale=2.0), _randn(gen, B, H, S, D)
        idx = torch.full((B, off[-1]), -1, dtype=torch.int32, device="cuda")
        for b in range(B):
            for h, n in enumerate(kept):
                idx[b, off[h]:off[h] + n] = _rows_of(n, S, gen)
        st.update(idx=idx, kept=kept, off=off, kl=(ctypes.c_int32 * H)(*kept),
                  pos=torch.full((B, off[-1]), -1, dtype=torch.int32, device="cuda"),
                  cache=torch.zeros((B, off[-1] // 16, 18 * D), dtype=torch.uint8, device="cuda"),
                  k_out=torch.empty((B * sum(kept), D), dtype=torch.bfloat16, device="cuda"),
                  v_out=torch.empty((B * sum(kept), D), dtype=torch.bfloat16, device="cuda"))
    else:
        T = c["T"]
        kept, off, cache, pos, rows, age, S0 = _cache(c, gen, T)
        new = S0 + age[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)   # positions of the new tokens
        st.update(kept=kept, off=off, cache=cache, pos=pos, rows=rows, new_pos=new.contiguous())
        if c["op"] == "append":
            st["k"], st["v"] = _randn(gen, B, H, T, D, scale=2.0), _randn(gen, B, H, T, D)
            st["nrows"] = (ctypes.c_int32 * H)(*([T] * H))
            st["k_out"] = torch.empty((B, H, T, D), dtype=torch.bfloat16, device="cuda")
            st["v_out"] = torch.empty((B, H, T, D), dtype=torch.bfloat16, device="cuda")
        else:
            st["q"] = _randn(gen, B, c["H_q"], T, D, scale=1.5)
            st["out"] = torch.empty((B, c["H_q"], T, D), dtype=torch.bfloat16, device="cuda")
            st["lse"] = torch.empty((B, c["H_q"], T), dtype=torch.float32, device="cuda")
    st["slot"] = (ctypes.c_int64 * (H + 1))(*st["off"])
    return st


# ------------------------------------------------- the 4-bit rows, plain form
def quantise(x):
    """x [..., D] -> (codes uint8 [..., D], scales e4m3 bytes [..., D/16]).  Per 16
    values: scale = amax / 6 rounded to e4m3, code = x / scale rounded to e2m1, both
    to nearest even and saturating.  The products below are exact in 32 bits."""
    g = x.float().unflatten(-1, (-1, 16))
    a = g.abs()
    top = a.amax(-1)
    s8 = (top / torch.full_like(top, 6.0)).clamp(max=448).to(torch.float8_e4m3fn)   # by a tensor: a true division
    s = s8.float()[..., None]
    code = ((a > 0.25 * s).byte() + (a >= 0.75 * s).byte() + (a > 1.25 * s).byte() + (a >= 1.75 * s).byte()
            + (a > 2.5 * s).byte() + (a >= 3.5 * s).byte() + (a > 5.0 * s).byte())
    code = torch.where(s > 0, code + 8 * torch.signbit(g).byte(), torch.zeros_like(code))
    return code.flatten(-2), s8.view(torch.uint8)


def values(code, s8):
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=code.device)
    v = lut[code.int()].unflatten(-1, (-1, 16)) * s8.view(torch.float8_e4m3fn).float()[..., None]
    return v.flatten(-2)


def pack(k, v):
    """Codes and scales of R rows (R a multiple of 16) -> [..., R/16, 18 D] bytes."""
    (kc, ks), (vc, vs) = k, v
    lead, (R, D) = kc.shape[:-2], kc.shape[-2:]
    kc = kc.reshape(*lead, R // 16, 16, 4, 2, D // 8)                 # row, quarter, half, byte
    kc = kc[..., 0, :] | kc[..., 1, :] << 4
    vc = vc.reshape(*lead, R // 16, 2, 4, 2, 8, D // 8)               # half, pair, key of the pair, slice, byte
    vc = (vc[..., 0, :, :] | vc[..., 1, :, :] << 4).transpose(-3, -2)
    ks = ks.reshape(*lead, R // 16, 2, 8, 4, D // 64).movedim(-4, -2)
    vs = vs.reshape(*lead, R // 16, 2, 4, 2, D // 16).movedim(-1, -4).transpose(-3, -2)
    return torch.cat([x.reshape(*lead, R // 16, -1) for x in (kc, vc, ks, vs)], -1)


def unpack(cache):
    """The inverse of pack: ((codes, scales) of the keys, of the values)."""
    lead, (N, D) = cache.shape[:-2], (cache.shape[-2], cache.shape[-1] // 18)
    kc, vc, ks, vs = cache.split((8 * D, 8 * D, D, D), -1)
    kc = kc.reshape(*lead, N, 16, 4, D // 8)
    kc = torch.stack((kc & 15, kc >> 4), -2).reshape(*lead, N * 16, D)
    vc = vc.reshape(*lead, N, 2, 8, 4, D // 8).transpose(-3, -2)
    vc = torch.stack((vc & 15, vc >> 4), -3).reshape(*lead, N * 16, D)
    ks = ks.reshape(*lead, N, 8, 4, 2, D // 64).movedim(-2, -4).reshape(*lead, N * 16, D // 16)
    vs = vs.reshape(*lead, N, D // 16, 4, 2, 2).transpose(-3, -2).movedim(-4, -1).reshape(*lead, N * 16, D // 16)
    return (kc, ks), (vc, vs)


def _row_ids(st):
    """[H_kv, M] row of each head's i-th row in a batch element's block, and which i exist."""
    off = torch.tensor(st["off"], device="cuda")
    cap = off[1:] - off[:-1]
    i = torch.arange(max(st["off"][h + 1] - st["off"][h] for h in range(len(st["off"]) - 1)), device="cuda")
    return off[:-1, None] + torch.minimum(i[None, :], cap[:, None] - 1), i[None, :] < cap[:, None]


# ------------------------------------------------------------------ one pass
def _rotate(x, w, c, cos, sin):
    """x [B, T, H, D] -> [B, H, T, D]: norm per head, rotation, one rounding."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    R = c["R"]
    r = y[..., :R]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :R // 2], r[..., R // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if c["inter"] else torch.cat((a, b), -1)
    return torch.cat((r, y[..., R:]), -1).to(torch.bfloat16).transpose(1, 2)


def _run_rotate(st):
    c = st["c"]
    B, T, Hq, H, D, row0 = c["B"], c["T"], c["H_q"], c["H_kv"], c["D"], c["row0"]
    q, k, v = st["qkv"].split((Hq * D, H * D, H * D), -1)
    if own:
        from attention_score_kv_gb300 import kvc as K
        ld = st["qkv"].shape[-1]
        K.kvc_qk_norm_rope(q, k, v, B, T, Hq, H, D, ld, ld, ld, c["R"], int(c["inter"]), st["qw"], st["kw"], EPS,
                           st["inv_freq"], st["pos"], c["S"], row0, st["q_out"], st["k_act"], st["v_act"])
        return st["q_out"], st["k_act"], st["v_act"]
    # angles of far positions need 64 bits
    ang = st["pos"].double()[..., None] * st["inv_freq"].double()
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    st["q_out"].copy_(_rotate(q.unflatten(-1, (Hq, D)), st["qw"], c, cos, sin))
    st["k_act"][:, :, row0:row0 + T] = _rotate(k.unflatten(-1, (H, D)), st["kw"], c, cos, sin)
    st["v_act"][:, :, row0:row0 + T] = v.unflatten(-1, (H, D)).transpose(1, 2)
    return st["q_out"], st["k_act"], st["v_act"]


def _run_gather(st):
    c = st["c"]
    B, H, S, D = c["B"], c["H_kv"], c["S"], c["D"]
    if own:
        from attention_score_kv_gb300 import kvc as K
        K.kvc_gather_q4(st["k"], st["v"], st["idx"], B, H, S, D, st["kl"], st["slot"], st["cache"], st["pos"])
        K.kvc_read_q4(st["cache"], B, H, D, st["slot"], None, st["kl"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"], st["pos"]
    kept, off = torch.tensor(st["kept"], device="cuda"), torch.tensor(st["off"], device="cuda")
    h = torch.repeat_interleave(torch.arange(H, device="cuda"), kept, output_size=sum(st["kept"]))
    row = torch.arange(sum(st["kept"]), device="cuda") + (off[:-1] - (kept.cumsum(0) - kept))[h]
    at = st["idx"][:, row].long()                                     # [B, T]
    st["pos"][:, row] = at.to(torch.int32)
    flat = ((torch.arange(B, device="cuda")[:, None] * H + h) * S + at).flatten()
    k, v = (values(*quantise(x.view(-1, D)[flat])).to(torch.bfloat16) for x in (st["k"], st["v"]))
    return k, v, st["pos"]


def _run_append(st):
    c = st["c"]
    B, H, T, D = c["B"], c["H_kv"], c["T"], c["D"]
    if own:
        from attention_score_kv_gb300 import kvc as K
        K.kvc_append_q4(st["k"], st["v"], st["new_pos"], B, H, T, D, st["slot"], st["rows"], st["cache"], st["pos"])
        K.kvc_read_q4(st["cache"], B, H, D, st["slot"], st["rows"], st["nrows"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"], st["pos"]
    t = torch.arange(T, device="cuda")
    off = torch.tensor(st["off"], device="cuda")
    row = (off[:-1] + st["rows"])[..., None] + t                      # [B, H, T]
    st["pos"].scatter_(1, row.flatten(1), st["new_pos"][:, None].expand(B, H, T).flatten(1))
    k, v = (values(*quantise(x)).to(torch.bfloat16) for x in (st["k"], st["v"]))
    return k, v, st["pos"]


def _run_attend(st):
    c = st["c"]
    B, T, Hq, H, D = c["B"], c["T"], c["H_q"], c["H_kv"], c["D"]
    if own:
        from attention_score_kv_gb300 import kvc as K
        if "ws" not in st:
            st["ws"] = K.attention_q4_workspace(B, T, Hq, H, D)
        K.kvc_attention_q4(st["q"], st["cache"], st["pos"], st["rows"], T, st["new_pos"], B, T, Hq, H, D, st["slot"],
                           st["out"], st["lse"], st["ws"])
        return st["out"], st["lse"]
    ids, real = _row_ids(st)
    k, v = (values(*x)[:, ids] for x in unpack(st["cache"]))          # [B, H, M, D]
    pos = st["pos"][:, ids]
    i = torch.arange(ids.shape[1], device="cuda")
    there = real & (i < (st["rows"] + T)[..., None]) & (pos >= 0)     # [B, H, M]
    see = there[:, :, None] & (pos[:, :, None] <= st["new_pos"][:, None, :, None])    # [B, H, T, M]
    q = st["q"].float().view(B, H, Hq // H, T, D)
    x = (q.flatten(2, 3) @ k.transpose(-1, -2)).view(B, H, -1, T, ids.shape[1]) / math.sqrt(D)
    x = x.masked_fill(~see[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(B, H, -1, T, D) / torch.where(z > 0, z, torch.ones_like(z))
    lse = torch.where(z > 0, m + torch.log(z), torch.full_like(z, -math.inf))
    return o.to(torch.bfloat16).view(B, Hq, T, D), lse.view(B, Hq, T)


def run(state):
    return {"rotate": _run_rotate, "gather": _run_gather, "append": _run_append, "attend": _run_attend}[
        state["c"]["op"]](state)


# ------------------------------------------------------------------ the floors
def work(case):
    c = case
    B, D, H = c["B"], c["D"], c["H_kv"]
    row = D * 9 // 8                       # bytes of a row's keys and values in the cache: 4.5 bits each value
    if c["op"] == "rotate":
        n = B * c["T"]
        return {"bytes": 2 * 2 * n * (c["H_q"] + 2 * H) * D + 4 * n + 2 * c["R"], "flops": 6 * n * (c["H_q"] + H) * D}
    if c["op"] == "gather":
        n = B * sum(_kept(c))              # read K and V, write the 4-bit rows, read them and write them out
        return {"bytes": n * (4 * D + 2 * row + 4 * D + 8), "flops": 8 * n * D}
    if c["op"] == "append":
        n = B * H * c["T"]
        return {"bytes": n * (4 * D + 2 * row + 4 * D + 8), "flops": 8 * n * D}
    kept, T = _kept(c), c["T"]
    rows = B * sum(n + (1 + max(kept) // 8) // 2 + T for n in kept)   # a sequence is half of its room old on average
    return {"bytes": rows * (row + 4) + 2 * B * T * c["H_q"] * D * 2 + 4 * B * T * c["H_q"],
            "flops": 4 * rows * (c["H_q"] // H) * T * D - 2 * B * c["H_q"] * T * (T - 1) * D}


# ----------------------------------------------------- the definition, 64 bits
def _exact_values(x):
    """Nearest e2m1 multiple of the group's scale, by distance, in 64 bits."""
    g = x.double().unflatten(-1, (-1, 16))
    a = g.abs()
    top = a.amax(-1, keepdim=True)
    want = (top / torch.full_like(top, 6.0)).clamp(max=448.0)
    # the 127 finite e4m3 values upward; nearest, ties to the even one (python's powers of two are exact)
    e4m3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16)
                                                             for m in range(8)][:119], dtype=torch.float64).to(x.device)
    up = torch.searchsorted(e4m3, want.contiguous()).clamp(min=1, max=126)       # e4m3[up - 1] < want <= e4m3[up]
    over, under = e4m3[up] - want, want - e4m3[up - 1]
    s = e4m3[torch.where((over < under) | ((over == under) & (up % 2 == 0)), up, up - 1)]
    level = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    d = [(a - lv * s).abs() for lv in level]
    best, at = d[0], torch.zeros_like(a, dtype=torch.int64)
    for n in range(1, 8):
        better = (d[n] < best) | ((d[n] == best) & (n % 2 == 0))
        best, at = torch.where(better, d[n], best), torch.where(better, torch.full_like(at, n), at)
    return (torch.sign(g) * level[at] * s).flatten(-2)


def _exact_rows(st, b, h, n):
    """The first n rows of head h of sequence b, straight from the bytes."""
    D, r0 = st["c"]["D"], st["off"][h]
    by = st["cache"][b]
    r = torch.arange(n, device="cuda")[:, None]
    d = torch.arange(D, device="cuda")[None, :]
    blk, i = (r0 + r) // 16, (r0 + r) % 16
    q, o = d // (D // 4), d % (D // 4)
    kn = by[blk, i * (D // 2) + q * (D // 8) + o % (D // 8)].long() >> 4 * (o // (D // 8))
    sl, o = d // (D // 8), d % (D // 8)
    vn = by[blk, 8 * D + (((i // 8) * 8 + sl) * 4 + (i % 8) // 2) * (D // 8) + o].long() >> 4 * (i % 2)
    g = d // 16
    kw = D // 64
    kb = by[blk, 16 * D + (((i % 8) * 4 + g // kw) * 2 + i // 8) * kw + g % kw].long()
    vb = by[blk, 17 * D + ((g * 4 + (i % 8) // 2) * 2 + i // 8) * 2 + i % 2].long()

    def val(nib, sb):
        nib = nib & 15
        e, m = (nib >> 1) & 3, (nib & 1).double()
        mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
        se, sm = (sb >> 3) & 15, (sb & 7).double()
        sc = torch.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8) * torch.exp2(se.double() - 7))
        return torch.where(nib >= 8, -mag, mag) * sc

    return val(kn, kb), val(vn, vb)


def exact(case, seed):
    st = prepare(case, seed)
    c = st["c"]
    B, D, H = c["B"], c["D"], c["H_kv"]
    if c["op"] == "rotate":
        T, Hq, R, row0 = c["T"], c["H_q"], c["R"], c["row0"]
        x = st["qkv"].double().view(B, T, Hq + 2 * H, D)
        ang = torch.einsum("bt,f->btf", st["pos"].double(), st["inv_freq"].double())[:, :, None]
        turn = torch.polar(torch.ones_like(ang), ang)

        def rot(y, w):
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + EPS) * w.double()
            lo = torch.arange(R // 2, device="cuda") * (2 if c["inter"] else 1)
            hi = lo + (1 if c["inter"] else R // 2)
            z = torch.complex(y[..., lo], y[..., hi]) * turn
            y = y.clone()
            y[..., lo], y[..., hi] = z.real, z.imag
            return y.permute(0, 2, 1, 3)

        k_act, v_act = st["k_act"].double(), st["v_act"].double()
        k_act[:, :, row0:row0 + T] = rot(x[:, :, Hq:Hq + H], st["kw"])
        v_act[:, :, row0:row0 + T] = x[:, :, Hq + H:].permute(0, 2, 1, 3)
        return rot(x[:, :, :Hq], st["qw"]).contiguous(), k_act, v_act
    if c["op"] == "gather":
        out = []
        for t in (st["k"], st["v"]):
            rows = [t[b, h, st["idx"][b, st["off"][h]:st["off"][h] + n].long()]
                    for b in range(B) for h, n in enumerate(st["kept"])]
            out.append(_exact_values(torch.cat(rows)))
        return out[0], out[1], None
    if c["op"] == "append":
        return _exact_values(st["k"]), _exact_values(st["v"]), None
    T, Hq = c["T"], c["H_q"]
    G = Hq // H
    out = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Hq, T), dtype=torch.float64, device="cuda")
    rows = st["rows"].tolist()
    for b in range(B):
        for h in range(H):
            n = rows[b][h] + T
            k, v = _exact_rows(st, b, h, n)
            pos = st["pos"][b, st["off"][h]:st["off"][h] + n]
            see = (pos >= 0)[None] & (pos[None] <= st["new_pos"][b][:, None])
            for g in range(G):
                x = st["q"][b, h * G + g].double() @ k.T / math.sqrt(D)
                x = x.masked_fill(~see, -math.inf)
                out[b, h * G + g] = torch.softmax(x, -1) @ v
                lse[b, h * G + g] = torch.logsumexp(x, -1)
    return out, lse
