"""The barriers of the many-row 4-bit attention, played through on the CPU.

The kernel's warps hand tiles to one another over mbarriers, and a wait looks at
the parity of a phase alone: a barrier that runs two phases ahead of a warp that
still waits for the first reads as not done.  Here the waits and arrivals of
every role are taken from the kernel's source, with their slots and phases, and
played in many orders, each role held back as long as the others can go on among
them.  No order may leave a warp waiting, and no tile of codes, operands, scores
or weights may be overwritten before its readers are through."""

import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_score_kv_gb300", "csrc",
                   "kvc_q4_attend_tc.cu")
OP = re.compile(r"(poll3?|\bwait|mbar_arrive|mbar_arrive_expect_tx|mma_commit|drain_wait)\(")
BAR = re.compile(r"&bars(?:->|\.)(\w+)(?:\[(.+?)\])?\)?$")


def split_args(text, at):
    """The arguments of the call whose opening parenthesis is at text[at]."""
    depth, start, out = 0, at + 1, []
    for i in range(at, len(text)):
        depth += text[i] in "([{"
        depth -= text[i] in ")]}"
        if (text[i] == "," and depth == 1) or depth == 0:
            out.append(" ".join(text[start:i].split()))
            start = i + 1
        if depth == 0:
            return out
    raise AssertionError("unbalanced")


def body_of(text, head):
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += text[i] == "{"
        depth -= text[i] == "}"
        if depth == 0:
            return text[at:i]
    raise AssertionError("unbalanced")


def ops_of(body):
    """The role's waits (bar, slot, phase) and arrivals (bar, slot, None), in order; locals put in."""
    names = dict(re.findall(r"(\w+) = (\(*i [^;,]*)[;,]", body))
    names.update(re.findall(r"uint32_t (bar) = ([^;]*);", body))

    def full(x):
        for _ in range(3):
            x = re.sub(r"\b(st|rs|vst|ph|bar)\b", lambda m: f"({names[m[0]]})" if m[0] in names else m[0], x)
        return x

    def place(x):
        m = BAR.search(full(x).strip("()"))
        return m and (m[1], m[2] or "0")

    ops = []
    for m in OP.finditer(body):
        args = split_args(body, m.end() - 1)
        for k in range(0, len(args) - 1, 2) if m[1] in ("poll", "poll3", "wait") else (0,):
            to = place(args[k])
            if to and m[1] != "drain_wait":
                ops.append((*to, None if m[1].startswith("m") else full(args[k + 1])))
    return ops


def kernel():
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    const = {k: int(v) for k, v in re.findall(r"\b(kRaw|kV|kSeen|kCodeWarps) = (\d+)", text)}
    roles = {r: ops_of(body_of(text, h)) for r, h in (
        ("load", "bool load_warp("), ("code", "bool code_warp("), ("score", "bool score_warp("),
        ("out", "bool out_warp("))}
    soft = text[text.index("(warp & 3) < live_quarters"):text.index("kvc_attend_q4_tc_join_kernel")]
    roles["soft"] = ops_of(soft)
    counts = dict(re.findall(r"mbar_init\(smem_u32\(&bars\.(\w+)(?:\[i\])?\), (\w+)\)", text))
    return const, roles, counts


CONST, ROLES, COUNTS = kernel()


def value(text, i, n):
    return eval(text.replace("/", "//"), {}, {"i": i, "n": n, **CONST})


class Stuck(Exception):
    pass


def play(n, live_warps, pick, roles=ROLES, const=CONST):
    """All roles over n tiles; pick chooses among the agents that can go on."""
    want = {b: live_warps if c == "live_warps" else CONST.get(c) or int(c) for b, c in COUNTS.items()}
    done, left = {}, {}                       # phases completed, arrivals missing

    def arrive(bar):
        left[bar] = left.get(bar, want[bar[0]]) - 1
        if left[bar] == 0:
            done[bar], left[bar] = done.get(bar, 0) + 1, want[bar[0]]

    def over(bar, parity):
        return (done.get(bar, 0) & 1) != parity

    # what each step of a tile needs of other steps, beside what the barriers say
    count = {}

    def mark(what, i, need=()):
        for w, j, k in need:
            assert j < 0 or count.get((w, j), 0) == k, f"{what} of tile {i} before {w} of tile {j}"
        count[what, i] = count.get((what, i), 0) + 1

    C, S = const["kCodeWarps"], live_warps
    started = {
        "load": lambda i: mark("fetch", i, [("read codes", i - const["kRaw"], C), ("masked", i - const["kSeen"], S)]),
        "code": lambda i: mark("read codes", i, [("copy", i, 1), ("scores", i - 2, 1), ("output", i - const["kV"], 1)]),
        "score": lambda i: mark("start scores", i, [("converted", i, C), ("masked", i - 2, S)]),
        "out": lambda i: mark("start output", i, [("converted", i, C), ("weights", i, S), ("output", i - 1, 1)]),
    }
    flights = {}                              # agent -> tiles whose copy or product is under way, in order

    def agent(role, name):
        ops = roles[role]
        once = [o for o in ops if o[0] == "q_full"]
        loop = [o for o in ops if o[0] != "q_full" and "n - 1" not in o[1]]
        first_arrival = next(k for k, o in enumerate(loop) if o[2] is None)
        if role == "soft":
            arrive(("q_full", 0))
        for o in once if role != "soft" else ():
            yield (o[0], 0), value(o[2], 0, n) & 1
        for i in range(n):
            for k, (bar, slot, phase) in enumerate(loop):
                at = (bar, value(slot, i, n))
                if phase is not None:
                    if "i - 1" in slot and i == 0:
                        continue              # the first tile follows no other
                    yield at, value(phase, i, n) & 1
                    continue
                if k == first_arrival and role in started:
                    started[role](i)
                if role in ("load", "score", "out"):
                    flights.setdefault(name, []).append((at, i))
                    continue
                if role == "code" and k == first_arrival:
                    mark("converted", i)
                if role == "soft" and bar == "s_free":
                    mark("masked", i, [("scores", i, 1), ("fetch", i, 1)])
                if role == "soft" and bar == "p_full":
                    mark("weights", i, [("output", i - 1, 1)])
                arrive(at)
                yield None
        for bar, slot, phase in (o for o in ops if "n - 1" in o[1]):
            yield (bar, value(slot, 0, n)), value(phase, 0, n) & 1

    names = [("load", 0), ("score", 0), ("out", 0), *(("code", w) for w in range(C)), *(("soft", w) for w in range(S))]
    agents = {a: agent(a[0], a) for a in names}
    wants = {a: None for a in names}
    landed = {"load": "copy", "score": "scores", "out": "output"}
    while agents or any(flights.values()):
        ready = [a for a in agents if wants[a] is None or over(*wants[a])]
        ready += [("land", a) for a, f in flights.items() if f]
        if not ready:
            raise Stuck({a: wants[a] for a in agents})
        a = pick(ready)
        if a[0] == "land":
            at, i = flights[a[1]].pop(0)
            mark(landed[a[1][0]], i)
            arrive(at)
            continue
        try:
            wants[a] = next(agents[a])
        except StopIteration:
            del agents[a]


def orders():
    for late in ("load", "score", "out", "code", "soft", "land"):
        for early in ("load", "score", "out", "code", "soft", "land"):
            if late != early:
                yield f"{late} last, {early} first", lambda r, e=early, l=late: min(
                    r, key=lambda a: (a[0] == l) - (a[0] == e))
    for seed in range(40):
        rng = random.Random(seed)
        yield f"random {seed}", lambda r, g=rng: g.choice(r)
    for seed in range(40):                    # each agent held back for a while, by turns
        rng = random.Random(100 + seed)
        weight = {}

        def pick(r, g=rng, w=weight):
            if g.random() < 0.02:
                w.clear()
            return min(r, key=lambda a: w.setdefault(a, g.random()))

        yield f"turns {seed}", pick


def test_the_source_has_every_role():
    assert {r: len(o) > 1 for r, o in ROLES.items()} == dict.fromkeys(("load", "code", "score", "out", "soft"), True)
    used = {o[0] for ops in ROLES.values() for o in ops}
    assert used == set(COUNTS) - {"drain"}
    assert all(any(o[0] == b and o[2] is not None for ops in ROLES.values() for o in ops) for b in used)


@pytest.mark.parametrize("n", [1, 2, 3, 5, 13])
@pytest.mark.parametrize("live_warps", [2, 8])
def test_no_order_leaves_a_warp_waiting(n, live_warps):
    for name, pick in orders():
        try:
            play(n, live_warps, pick)
        except Stuck as e:
            raise AssertionError(f"{name}: {e}") from None


def test_a_barrier_that_runs_ahead_is_found():
    """The same check on a protocol whose outputs wait for the scores' two-slot barrier."""
    planted = [("k_full", "i & 1", "i >> 1"), ("p_full", "0", "i"), ("o_done", "i % kV", None)]
    with pytest.raises(Stuck):
        for _, pick in orders():
            play(13, 2, pick, roles={**ROLES, "out": planted})
