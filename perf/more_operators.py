"""Cases of the operators on both sides of the 8-bit retained cache: the cache
itself (gather into it, append to it, read it back), attention over it, and the
attention of a prompt chunk over the active layer's buffers, which comes before
the compress.  Both attentions take scores capped by a tanh and a bias by
distance; the chunk's takes a document mask or a prefix mask too.

``own`` False computes the plain forms with elementary torch operations;
``own`` True makes the calls of ``attention_score_kv_gb300.kvc``.

The 8-bit cache holds rows of e4m3 codes, keys and values apart, with one scale
each per block of 16 rows of a head: the smallest power of two (2^-100 at least)
that brings the block's values to 448 or less.
"""

import ctypes
import math

import torch

own = False

LEAST = 27               # biased exponent of the smallest scale, 2^-100


# ------------------------------------------------------------------ the cases
def listed():
    return [
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
             uneven=False, cap=0.0, bias=False),
        # One token of four requests over unequal budgets (Qwen2.5-14B layer), scores biased by distance.
        dict(name="attend one token, uneven, bias", op="attend", B=4, T=1, H_q=40, H_kv=8, D=128, keep=9830,
             uneven=True, cap=0.0, bias=True),
        # A full serving batch, one token each (Mistral-7B heads, budget 4096), scores capped.
        dict(name="attend 64 requests, cap", op="attend", B=64, T=1, H_q=32, H_kv=8, D=128, keep=4096, uneven=False,
             cap=30.0, bias=False),
        # The prompt of a follow-up turn: 512 new tokens over the retained rows and themselves.
        dict(name="attend a turn of 512", op="attend", B=1, T=512, H_q=32, H_kv=8, D=128, keep=4096, uneven=False,
             cap=0.0, bias=False),
        # The last token of a prompt that leaves one over, over 8K of the active layer.
        dict(name="chunk of one token over 8K", op="chunk", B=1, T=1, H_q=32, H_kv=8, S=8192, D=128, row0=8191,
             mask="causal", cap=0.0, bias=False),
        # A ragged batch of packed documents, head dim 64, scores biased by distance.
        dict(name="chunk of documents, bias", op="chunk", B=3, T=1537, H_q=40, H_kv=8, S=2048, D=64, row0=511,
             mask="documents", cap=0.0, bias=True),
        # The last prefill chunk of a Llama-3.1-8B layer at 8K, scores capped.
        dict(name="chunk of 2048 over 8K, cap", op="chunk", B=1, T=2048, H_q=32, H_kv=8, S=8192, D=128, row0=6144,
             mask="causal", cap=30.0, bias=False),
        # A prefill chunk at 32K (Mistral-7B heads) behind a prefix that all of its tokens see whole.
        dict(name="chunk of 2048 over 32K, prefix", op="chunk", B=1, T=2048, H_q=32, H_kv=8, S=32768, D=128,
             row0=30720, mask="prefix", cap=0.0, bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gather", "append", "attend", "attend", "chunk", "chunk"))
    D = rng.choice((64, 128, 128))
    H_kv = rng.choice((1, 2, 4, 8, 8))
    G = rng.choice((1, 2, 4, 5, 7, 8))
    if op == "gather":
        S = _log(rng, 128, 65536)
        keep = min(S, _log(rng, 16, 9830))
        B = max(1, min(_log(rng, 1, 8), 39320 // keep, 131072 // S))
        return dict(op=op, B=B, H_kv=H_kv, S=S, D=D, keep=keep, uneven=rng.random() < 0.5)
    if op == "chunk":
        T = rng.choice((1, rng.randrange(2, 33), _log(rng, 33, 2048), _log(rng, 33, 2048)))
        S = max(T, _log(rng, 128, 32768))
        B = max(1, min(_log(rng, 1, 64), 2 ** 21 // (S * H_kv), 2 ** 31 // (T * S * H_kv * G)))
        return dict(op=op, B=B, T=T, H_q=H_kv * G, H_kv=H_kv, S=S, D=D, row0=rng.choice((S - T, rng.randrange(0, S - T + 1))),
                    mask=rng.choice(("causal", "documents", "prefix")), cap=rng.choice((0.0, 0.0, 20.0, 50.0)),
                    bias=rng.random() < 0.3)
    keep = _log(rng, 16, 16384)
    if op == "append":
        B = max(1, min(_log(rng, 1, 64), 262144 // keep))
        return dict(op=op, B=B, H_kv=H_kv, T=rng.choice((1, 1, 2, 3, 5, 8, 17, 33)), D=D, keep=keep,
                    uneven=rng.random() < 0.3)
    T = rng.choice((1, 1, 1, 2, 3, 5, 8, _log(rng, 9, 512)))
    B = max(1, min(_log(rng, 1, 64), 262144 // keep, 2 * 10 ** 6 // (T * G * keep)))
    return dict(op=op, B=B, T=T, H_q=H_kv * G, H_kv=H_kv, D=D, keep=keep, uneven=rng.random() < 0.5,
                cap=rng.choice((0.0, 0.0, 20.0, 50.0)), bias=rng.random() < 0.3)


# ------------------------------------------------------------------ the inputs
def _kept(c):
    """Retained rows of each KV head: equal, or spread 1:3 around the mean."""
    H, keep = c["H_kv"], c["keep"]
    if not c["uneven"] or H == 1:
        return [keep] * H
    w = [1.0 / (0.25 + 0.5 * ((h * 5) % H) / (H - 1)) for h in range(H)]
    most = c.get("S", 1 << 30)
    return [max(min(16, most), min(most, int(keep * H * x / sum(w)))) for x in w]


def _slots(kept, extra):
    """First row of each head's slot (multiples of 16) and, last, a batch element's rows."""
    off = [0]
    for n in kept:
        off.append(off[-1] + (n + extra + 15) // 16 * 16)
    return off


def _rows_of(kept, S, gen):
    """Ascending positions of `kept` rows out of S."""
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
    k8, v8 = (torch.empty((B, R, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    scale = torch.empty((B, R // 16, 2), device="cuda")
    for b0 in range(0, B, 8):
        n = min(8, B - b0)
        for i, t in enumerate((k8, v8)):
            x = _randn(gen, n, R // 16, 16, D).float()
            s = scale_of(x.abs().amax((-1, -2)))
            scale[b0:b0 + n, :, i] = s
            t[b0:b0 + n] = codes(x, s[..., None, None]).view(torch.uint8).view(n, R, D)
    S0 = 4 * max(kept)
    age = torch.randint(0, room, (B,), generator=gen, device="cuda", dtype=torch.int32)   # tokens decoded so far
    pos = torch.full((B, R), -1, dtype=torch.int32, device="cuda")
    for h, n in enumerate(kept):
        r = torch.arange(off[h + 1] - off[h] - n, device="cuda", dtype=torch.int32)
        pos[:, off[h]:off[h] + n] = _rows_of(n, S0, gen)
        pos[:, off[h] + n:off[h + 1]] = S0 + r
    rows = torch.tensor(kept, dtype=torch.int32, device="cuda")[None, :] + age[:, None]
    return kept, off, k8, v8, scale, pos, rows, age, S0


def _slopes(c):
    """One slope per query head, 2^(-8 (h + 1) / H)."""
    H = c["H_q"]
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H) if c["bias"] else None


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = dict(c=c)
    D, B, H = c["D"], c["B"], c["H_kv"]
    if c["op"] == "chunk":
        T, S, row0 = c["T"], c["S"], c["row0"]
        st["q"] = _randn(gen, B, c["H_q"], T, D, scale=1.5)
        st["k"], st["v"] = _randn(gen, B, H, S, D), _randn(gen, B, H, S, D)
        t = torch.arange(T, device="cuda", dtype=torch.int32)
        # the sequences of a batch end at their own tokens; the padding behind sees nothing
        n = torch.randint(max(1, T - T // 4), T + 1, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        if B == 1:
            n = torch.full_like(n, T)
        pos = torch.where(t < n, row0 + t, -1)
        first = last = None
        if c["mask"] == "documents":           # a position starts a document, and positions see their own document
            starts = torch.rand((B, S), generator=gen, device="cuda") < 4.0 / (S + 4)
            at = torch.where(starts, torch.arange(S, device="cuda", dtype=torch.int32), 0).cummax(1).values
            first = torch.where(pos >= 0, at[:, row0:row0 + T], 0).to(torch.int32).contiguous()
        if c["mask"] == "prefix":              # the first positions see each other both ways
            front = torch.randint(row0, row0 + T + 1, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
            last = torch.maximum(pos, front - 1).contiguous()
        st.update(pos=pos.contiguous(), first=first, last=last, slopes=_slopes(c),
                  out=torch.empty((B, c["H_q"], T, D), dtype=torch.bfloat16, device="cuda"),
                  lse=torch.empty((B, c["H_q"], T), dtype=torch.float32, device="cuda"))
        return st
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
                  k8=torch.zeros((B, off[-1], D), dtype=torch.uint8, device="cuda"),
                  v8=torch.zeros((B, off[-1], D), dtype=torch.uint8, device="cuda"),
                  scale=torch.ones((B, off[-1] // 16, 2), device="cuda"),
                  k_out=torch.empty((B * sum(kept), D), dtype=torch.bfloat16, device="cuda"),
                  v_out=torch.empty((B * sum(kept), D), dtype=torch.bfloat16, device="cuda"))
    else:
        T = c["T"]
        kept, off, k8, v8, scale, pos, rows, age, S0 = _cache(c, gen, T)
        new = S0 + age[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)   # positions of the new tokens
        st.update(kept=kept, off=off, k8=k8, v8=v8, scale=scale, pos=pos, rows=rows, new_pos=new.contiguous())
        if c["op"] == "append":
            st["k"], st["v"] = _randn(gen, B, H, T, D, scale=2.0), _randn(gen, B, H, T, D)
            # read back with the block before, whose last rows may share a scale with the new ones
            st["first"], st["nrows"] = rows - 16, (ctypes.c_int32 * H)(*([T + 16] * H))
            st["k_out"] = torch.empty((B, H, T + 16, D), dtype=torch.bfloat16, device="cuda")
            st["v_out"] = torch.empty((B, H, T + 16, D), dtype=torch.bfloat16, device="cuda")
        else:
            st["slopes"] = _slopes(c)
            st["q"] = _randn(gen, B, c["H_q"], T, D, scale=1.5)
            st["out"] = torch.empty((B, c["H_q"], T, D), dtype=torch.bfloat16, device="cuda")
            st["lse"] = torch.empty((B, c["H_q"], T), dtype=torch.float32, device="cuda")
    st["slot"] = (ctypes.c_int64 * (H + 1))(*st["off"])
    return st


# ------------------------------------------------- the 8-bit rows, plain form
def scale_of(top):
    """The scale of a block whose largest magnitude is `top` (fp32): its exponent, one
    more where the significand is above 1.75, less the 8 of 448 = 1.75 * 2^8."""
    e = ((top.view(torch.int32) + 0x1fffff) >> 23) - 8
    return (e.clamp(min=LEAST) << 23).view(torch.float32)


def codes(x, scale):
    return (x / scale).to(torch.float8_e4m3fn)          # an exact quotient, one rounding


def held(x, scale):
    return codes(x, scale).float() * scale


def _row_ids(st):
    """[H_kv, M] row of each head's i-th row in a batch element's block, and which i exist."""
    off = torch.tensor(st["off"], device="cuda")
    cap = off[1:] - off[:-1]
    i = torch.arange(max(st["off"][h + 1] - st["off"][h] for h in range(len(st["off"]) - 1)), device="cuda")
    return off[:-1, None] + torch.minimum(i[None, :], cap[:, None] - 1), i[None, :] < cap[:, None]


def _values(st, i):
    """All rows of the cache's keys (i = 0) or values (1), fp32."""
    codes8 = (st["k8"], st["v8"])[i].view(torch.float8_e4m3fn).float()
    return codes8 * st["scale"][..., i].repeat_interleave(16, 1)[..., None]


# ------------------------------------------------------------------ one pass
def _run_gather(st):
    c = st["c"]
    B, H, S, D = c["B"], c["H_kv"], c["S"], c["D"]
    if own:
        from attention_score_kv_gb300 import kvc as K
        K.kvc_gather_q8(st["k"], st["v"], st["idx"], B, H, S, D, st["kl"], st["slot"], st["k8"], st["v8"],
                        st["scale"], st["pos"])
        K.kvc_read_q8(st["k8"], st["v8"], st["scale"], B, H, D, st["slot"], None, st["kl"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"], st["pos"]
    kept, off = torch.tensor(st["kept"], device="cuda"), torch.tensor(st["off"], device="cuda")
    h = torch.repeat_interleave(torch.arange(H, device="cuda"), kept, output_size=sum(st["kept"]))
    row = torch.arange(sum(st["kept"]), device="cuda") + (off[:-1] - (kept.cumsum(0) - kept))[h]
    at = st["idx"][:, row].long()                                     # [B, rows]
    st["pos"][:, row] = at.to(torch.int32)
    flat = ((torch.arange(B, device="cuda")[:, None] * H + h) * S + at).flatten()
    out = []
    for t in (st["k"], st["v"]):
        x = torch.zeros((B, st["off"][-1], D), device="cuda")
        x[:, row] = t.view(-1, D)[flat].float().view(B, -1, D)
        x = x.view(B, -1, 16, D)
        x = held(x, scale_of(x.abs().amax((-1, -2)))[..., None, None])
        out.append(x.view(B, -1, D)[:, row].to(torch.bfloat16).view(-1, D))
    return out[0], out[1], st["pos"]


def _run_append(st):
    c = st["c"]
    B, H, T, D = c["B"], c["H_kv"], c["T"], c["D"]
    if own:
        from attention_score_kv_gb300 import kvc as K
        K.kvc_append_q8(st["k"], st["v"], st["new_pos"], B, H, T, D, st["slot"], st["rows"], st["k8"], st["v8"],
                        st["scale"], st["pos"])
        K.kvc_read_q8(st["k8"], st["v8"], st["scale"], B, H, D, st["slot"], st["first"], st["nrows"], st["k_out"],
                      st["v_out"])
        return st["k_out"], st["v_out"], st["pos"]
    off = torch.tensor(st["off"], device="cuda")
    n0 = st["rows"].long()                                            # [B, H]
    t = torch.arange(T, device="cuda")
    row = (off[:-1] + n0)[..., None] + t
    st["pos"].scatter_(1, row.flatten(1), st["new_pos"][:, None].expand(B, H, T).flatten(1))
    # the block before the one that the cache ends in, that one, and those that the new rows reach
    blk0 = n0 // 16 - 1
    nb = 2 + (T + 14) // 16
    blk = (off[:-1] // 16 + blk0)[..., None] + torch.arange(nb, device="cuda")     # [B, H, nb] of the batch element
    blk = blk.clamp(max=st["off"][-1] // 16 - 1)
    at = torch.arange(nb * 16, device="cuda") + (blk0 * 16 - n0)[..., None]        # token of a row; < 0: held before
    old, new = at < 0, (at >= 0) & (at < T)
    b = torch.arange(B, device="cuda")[:, None, None]
    out = []
    for i, (t8, x) in enumerate(((st["k8"], st["k"]), (st["v8"], st["v"]))):
        s_old = st["scale"][..., i][b, blk]                                        # [B, H, nb]
        was = t8.view(B, -1, 16, D)[b, blk].view(torch.float8_e4m3fn).float() * s_old[..., None, None]
        take = at.clamp(0, T - 1)[..., None].expand(B, H, nb * 16, D)
        now = torch.gather(x.float(), 2, take) * new[..., None]
        need = scale_of(now.view(B, H, nb, 16, D).abs().amax((-1, -2)))
        s = torch.where(old.view(B, H, nb, 16).any(-1), torch.maximum(need, s_old), need)
        rows = torch.where(old[..., None], was.view(B, H, nb * 16, D), now).view(B, H, nb, 16, D)
        rows = held(rows, s[..., None, None]).view(B, H, nb * 16, D)
        pick = torch.arange(-16, T, device="cuda") + (n0 - blk0 * 16)[..., None]
        out.append(torch.gather(rows, 2, pick[..., None].expand(B, H, T + 16, D)).to(torch.bfloat16))
    return out[0], out[1], st["pos"]


def _softmax_of(x, see, v, shape):
    """Scores [.., Q, M] (changed in place), which of them count, values -> output, log of the sum."""
    x.masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(shape) / torch.where(z > 0, z, torch.ones_like(z))
    lse = torch.where(z > 0, m + torch.log(z), torch.full_like(z, -math.inf))
    return o.to(torch.bfloat16), lse


def _scores(c, q, k, slopes, far):
    """Scores [B, H_kv, G, T, M]: the product, capped, less the slope times the distance `far`."""
    B, T, Hq, H, D = c["B"], c["T"], c["H_q"], c["H_kv"], c["D"]
    x = (q.float().view(B, H, -1, D) @ k.transpose(-1, -2)).view(B, H, Hq // H, T, -1).div_(math.sqrt(D))
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    if slopes is not None:
        x.sub_(slopes.view(1, H, -1, 1, 1) * far)
    return x


def _run_attend(st):
    c = st["c"]
    B, T, Hq, H, D = c["B"], c["T"], c["H_q"], c["H_kv"], c["D"]
    if own:
        from attention_score_kv_gb300 import kvc as K
        if "ws" not in st:
            st["ws"] = K.attention_q8_workspace(B, T, Hq, H, D)
        K.kvc_attention_q8(st["q"], st["k8"], st["v8"], st["scale"], st["pos"], st["rows"], T, st["new_pos"], B, T, Hq,
                           H, D, st["slot"], c["cap"], st["slopes"], st["out"], st["lse"], st["ws"])
        return st["out"], st["lse"]
    ids, real = _row_ids(st)
    pos = st["pos"][:, ids]
    i = torch.arange(ids.shape[1], device="cuda")
    there = real & (i < (st["rows"] + T)[..., None]) & (pos >= 0)     # [B, H, M]
    see = there[:, :, None] & (pos[:, :, None] <= st["new_pos"][:, None, :, None])    # [B, H, T, M]
    far = (st["new_pos"][:, None, :, None] - pos[:, :, None])[:, :, None].float()
    x = _scores(c, st["q"], _values(st, 0)[:, ids], st["slopes"], far)
    o, lse = _softmax_of(x, see[:, :, None], _values(st, 1)[:, ids], (B, H, Hq // H, T, D))
    return o.view(B, Hq, T, D), lse.view(B, Hq, T)


def _run_chunk(st):
    c = st["c"]
    B, T, Hq, H, S, D = c["B"], c["T"], c["H_q"], c["H_kv"], c["S"], c["D"]
    if own:
        from attention_score_kv_gb300 import kvc as K
        if "ws" not in st:
            st["ws"] = K.attention_chunk_workspace(B, T, Hq, H, D)
        K.kvc_attention_chunk(st["q"], st["k"], st["v"], st["pos"], st["first"], st["last"], B, T, Hq, H, S, D,
                              c["cap"], st["slopes"], st["out"], st["lse"], st["ws"])
        return st["out"], st["lse"]
    j = torch.arange(S, device="cuda", dtype=torch.int32)
    pos = st["pos"][:, None, None, :, None]                           # [B, 1, 1, T, 1]
    last = pos if st["last"] is None else st["last"][:, None, None, :, None]
    see = (j <= last) & (pos >= 0)
    if st["first"] is not None:
        see &= j >= st["first"][:, None, None, :, None]
    x = _scores(c, st["q"], st["k"].float(), st["slopes"], (pos - j).abs().float())
    o, lse = _softmax_of(x, see, st["v"].float(), (B, H, Hq // H, T, D))
    return o.view(B, Hq, T, D), lse.view(B, Hq, T)


def run(state):
    return {"gather": _run_gather, "append": _run_append, "attend": _run_attend, "chunk": _run_chunk}[
        state["c"]["op"]](state)


# ------------------------------------------------------------------ the floors
def work(case):
    c = case
    B, D, H = c["B"], c["D"], c["H_kv"]
    if c["op"] == "gather":
        n = B * sum(_kept(c))              # read K and V, write the 8-bit rows, read them and write them out
        return {"bytes": n * (4 * D + 2 * (2 * D) + 4 * D + 1 + 8), "flops": 8 * n * D}
    if c["op"] == "append":
        n = B * H * c["T"]                 # and 16 rows more that are read back
        return {"bytes": n * (4 * D + 2 * D + 8) + B * H * (c["T"] + 16) * 6 * D, "flops": 8 * n * D}
    T, Hq = c["T"], c["H_q"]
    if c["op"] == "chunk":
        # pairs and keys that a causal chunk sees; a document a third or so of that, a prefix on average T^2 / 6 more
        row0 = c["row0"]
        share = 0.3 if c["mask"] == "documents" else 1.0
        pairs = (T * row0 + T * (T + 1) // 2 + (T * T // 6 if c["mask"] == "prefix" else 0)) * share
        pairs *= 1.0 if B == 1 else 0.875
        keys = (row0 + T) * (1.0 if T > 1 else share)
        return {"bytes": int(B * H * keys * 4 * D + B * Hq * T * (4 * D + 4)), "flops": int(4 * B * Hq * D * pairs)}
    kept = _kept(c)
    rows = B * sum(n + (1 + max(kept) // 8) // 2 + T for n in kept)   # a sequence is half of its room old on average
    return {"bytes": int(rows * (2 * D + 4.5)) + B * T * Hq * (4 * D + 4),
            "flops": 4 * rows * (Hq // H) * T * D - 2 * B * Hq * T * (T - 1) * D}


# ----------------------------------------------------- the definition, 64 bits
def _grid(device):
    """The e4m3 values from 0 to 448, ascending."""
    v = [m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64).to(device)


def _exact_held(x, scale):
    """Nearest multiple of the scale by an e4m3 value, ties to the even one; x fp64."""
    grid = _grid(x.device)
    a = x.abs() / scale
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    take = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[take] * scale, x)


def _exact_scale(top):
    """2^k, k the least integer with top <= 448 * 2^k, at least -100."""
    m, e = torch.frexp(top / 448.0)
    k = torch.where(m == 0.5, e - 1, e).clamp(min=-100)
    return torch.exp2(torch.where(top > 0, k, torch.full_like(k, -100)).double())


def _exact_byte(by):
    e, m = (by >> 3) & 15, (by & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(by >= 128, -v, v)


def _exact_rows(st, b, h, r):
    """Rows r of head h of sequence b: keys and values, straight from the bytes."""
    at = st["off"][h] + r
    s = st["scale"][b, at // 16].double()
    return (_exact_byte(st["k8"][b, at].long()) * s[:, :1], _exact_byte(st["v8"][b, at].long()) * s[:, 1:])


def _exact_attention(q, k, v, see, cap, bias):
    """One head: q [T, D], k and v [M, D], see [T, M], bias [T, M] or None, all in 64 bits."""
    x = q @ k.T / math.sqrt(q.shape[1])
    if cap:
        x = cap * torch.tanh(x / cap)
    if bias is not None:
        x = x + bias
    x = x.masked_fill(~see, -math.inf)
    some = see.any(-1, keepdim=True)
    return torch.softmax(x, -1).masked_fill(~some, 0.0) @ v, torch.logsumexp(x, -1)


def exact(case, seed):
    st = prepare(case, seed)
    c = st["c"]
    B, D, H = c["B"], c["D"], c["H_kv"]
    if c["op"] == "gather":
        out = []
        for t in (st["k"], st["v"]):
            rows = []
            for b in range(B):
                for h, n in enumerate(st["kept"]):
                    x = t[b, h, st["idx"][b, st["off"][h]:st["off"][h] + n].long()].double()
                    y = torch.cat((x, x.new_zeros((-n % 16, D)))).view(-1, 16 * D)
                    y = _exact_held(y, _exact_scale(y.abs().amax(-1, keepdim=True)))
                    rows.append(y.view(-1, D)[:n])
            out.append(torch.cat(rows))
        return out[0], out[1], None
    if c["op"] == "append":
        T = c["T"]
        out = [torch.empty((B, H, T + 16, D), dtype=torch.float64, device="cuda") for _ in range(2)]
        n0s = st["rows"].tolist()
        for b in range(B):
            for h in range(H):
                n0 = n0s[b][h]
                lo = n0 - 16 - n0 % 16                                # a block's first row
                was = _exact_rows(st, b, h, torch.arange(lo, n0, device="cuda"))
                for i, x in enumerate((st["k"], st["v"])):
                    y = torch.cat((was[i], x[b, h].double()))
                    y = torch.cat((y, y.new_zeros((-len(y) % 16, D)))).view(-1, 16, D)
                    new = torch.arange(lo, lo + y.shape[0] * 16, device="cuda").view(-1, 16, 1) >= n0
                    s = _exact_scale((y * new).abs().amax((1, 2)))
                    s_old = st["scale"][b, (st["off"][h] + lo) // 16:][:len(s), i].double()
                    s = torch.where(new[:, 0, 0], s, torch.maximum(s, s_old))
                    y = _exact_held(y.flatten(1), s[:, None]).view(-1, D)
                    out[i][b, h] = y[n0 - 16 - lo:n0 + T - lo]
        return out[0], out[1], None
    T, Hq = c["T"], c["H_q"]
    G = Hq // H
    out = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Hq, T), dtype=torch.float64, device="cuda")
    slopes = None if st["slopes"] is None else st["slopes"].double()
    rows = st["rows"].tolist() if c["op"] == "attend" else None
    for b in range(B):
        for h in range(H):
            if c["op"] == "attend":
                n = rows[b][h] + T
                k, v = _exact_rows(st, b, h, torch.arange(n, device="cuda"))
                pos, qp = st["pos"][b, st["off"][h]:st["off"][h] + n].double(), st["new_pos"][b].double()
                see = (pos >= 0)[None] & (pos[None] <= qp[:, None])
            else:
                k, v = st["k"][b, h].double(), st["v"][b, h].double()
                pos, qp = torch.arange(c["S"], device="cuda", dtype=torch.float64), st["pos"][b].double()
                hi = qp if st["last"] is None else st["last"][b].double()
                see = (pos[None] <= hi[:, None]) & (qp >= 0)[:, None]
                if st["first"] is not None:
                    see = see & (pos[None] >= st["first"][b].double()[:, None])
            for g in range(h * G, h * G + G):
                bias = None if slopes is None else -slopes[g] * (qp[:, None] - pos[None]).abs()
                out[b, g], lse[b, g] = _exact_attention(st["q"][b, g].double(), k, v, see, c["cap"], bias)
    return out, lse
