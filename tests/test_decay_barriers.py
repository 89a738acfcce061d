"""The mbarrier protocol of the decayed tensor-core prefill, run on the CPU.

A wait by parity tells neighbouring phases apart and no others: a warp that
waits for a phase while the barrier can complete the next one too may find the
parity of a phase that is still open, and wait for itself.  The roles of
``prefill_decay.cuh`` are stepped here as 16 agents (TMA thread, three MMA
threads, 4 P, 4 state, 4 output warps) whose barriers, guards, parities and
arrival counts are read from the source; every agent is held back at every one of
its steps until the others can do no more.  All chunks have to be finished, and
no wait may pass before the chunk that it is for.
"""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_linear_b200", "csrc",
                   "prefill_decay.cuh")
ITEMS = [2, 1, 4]  # chunks of the items that the CTA works on


def _args(text, at):
    """The comma-separated arguments of the parenthesis that opens at text[at]."""
    depth, start, out = 0, at + 1, []
    for i in range(at, len(text)):
        c = text[i]
        depth += c in "([{"
        depth -= c in ")]}"
        if (c == "," and depth == 1) or depth == 0:
            out.append(text[start:i].strip())
            start = i + 1
        if depth == 0:
            return out
    raise AssertionError("unbalanced")


def _expr(text):
    """A C expression over integers as a function of a dict of its variables."""
    m = re.fullmatch(r"(.*?)\?(.*):(.*)", text)
    if m:
        text = f"({m[2]}) if ({m[1]}) else ({m[3]})"
    code = compile(text.strip().replace("&&", " and ").replace("||", " or "), "<source>", "eval")
    return lambda env: int(eval(code, {"__builtins__": {}}, dict(env)))


def _barrier(text):
    m = re.fullmatch(r"&?(\w+)(?:\[(.*)\])?", text)
    return m[1], _expr(m[2] or "0")


class Ops:
    """The waits and arrivals of one role's part of the kernel, by barrier name in order of appearance."""

    def __init__(self, text):
        self.waits, self.arrivals = {}, {}
        for m in re.finditer(r"(?<![\w.:])(?:warp_)?wait\(|\b(?:mbar_arrive|mbar_arrive_expect_tx|mma_commit)\(", text):
            a = _args(text, m.end() - 1)
            name, index = _barrier(a[0])
            if "wait" in m[0]:
                lead = text[text.rfind("\n", 0, m.start()):m.start()]
                g = re.search(r"([gn]) > (\d) && !$", lead) or re.search(r"([gn]) == (\d) \|\| $", lead)
                first = 0 if g is None else int(g[2]) + 1
                var = None if g is None else g[1]
                self.waits.setdefault(name, []).append((index, _expr(a[1]), var, first))
            else:
                self.arrivals.setdefault(name, []).append(index)


@pytest.fixture(scope="module")
def kernel():
    text = open(SRC).read()
    body = text[text.index("prefill_decay_kernel(const __grid_constant__"):]
    init, parts = {}, re.split(r"// -{20,} (.+)\n", body)
    for m in re.finditer(r"mbar_init\(", parts[0]):
        a = _args(parts[0], m.end() - 1)
        init[_barrier(a[0])[0]] = _expr(a[1])
    roles = dict(zip(parts[1::2], parts[2::2]))
    mma = re.split(r"else if \(warp == WARP_MMA_B\)|\} else \{\n\s+constexpr uint32_t id_pv", roles.pop("MMA threads"))
    assert len(mma) == 3
    roles = {k: Ops(v) for k, v in (*roles.items(), ("A", mma[0]), ("B", mma[1]), ("C", mma[2]))}
    return init, roles


class Machine:
    def __init__(self, init, state_only):
        self.count = {k: v({"state_only": state_only, "i": 0}) for k, v in init.items()}
        self.bars = {}

    def bar(self, name, i):
        return self.bars.setdefault((name, i), [0, []])  # arrivals of the open phase, chunks of the complete ones

    def arrive(self, name, i, chunk):
        b = self.bar(name, i)
        b[0] += 1
        if b[0] == self.count[name]:
            b[0] = 0
            b[1].append(chunk)

    def done(self, name, i, parity):
        return (len(self.bar(name, i)[1]) & 1) != parity


def _chunks(state_only, tails):
    out, g = [], 0
    for r, nc in enumerate(ITEMS):
        for c in range(nc):
            out.append(dict(g=g, s=g & 1, n=g >> 1, r=r, first=c == 0, state_only=state_only, tail=tails and c == nc - 1))
            g += 1
    return out


def _agents(roles, state_only, tails):
    """Generators of ("wait", name, index, parity, chunk waited for) and ("arrive", name, index, chunk)."""
    chunks = _chunks(state_only, tails)

    def wait(role, name, env, chunk, nth=0):
        index, parity, var, first = roles[role].waits[name][nth]
        if var is None or env[var] >= first:
            yield "wait", name, index(env), parity(env), chunk

    def arrive(role, name, env, nth=0):
        yield "arrive", name, roles[role].arrivals[name][nth](env), env["g"]

    def tma():
        for e in chunks:
            for x in ("k", "v") if state_only else ("k", "v", "q"):
                yield from wait("TMA producer", x + "_empty", e, e["g"] - 2)
                yield from arrive("TMA producer", x + "_full", e)

    def mma_a():
        for e in chunks:
            yield from wait("A", "o_empty", e, e["g"] - 2)
            yield from wait("A", "q_full", e, e["g"])
            yield from wait("A", "k_full", e, e["g"])
            for x in ("p_full", "q_empty", "k_empty"):
                yield from arrive("A", x, e)

    def mma_b():
        for e in chunks:
            yield from wait("B", "k_full", e, e["g"])
            yield from wait("B", "ds_empty", e, e["g"] - 1)
            for qd in range(4):
                x = dict(e, qd=qd)
                yield from wait("B", "vt_full", x, e["g"])
                yield from arrive("B", "vt_empty", x)
            yield from arrive("B", "ds_full", e)
            yield from arrive("B", "k_empty", e)

    def mma_c():
        for e in chunks:
            yield from wait("C", "p_ready", e, e["g"])
            yield from arrive("C", "v_empty", e)
            yield from wait("C", "o_empty", e, e["g"] - 1)
            yield from wait("C", "s_full", e, e["g"])
            yield from arrive("C", "o_full", e)
            yield from arrive("C", "q_empty", e)

    def p_warp():
        for e in chunks:
            if e["first"]:
                yield "arrive", "tab_full", 0, e["r"]
                index, parity, _, _ = roles["P warps"].waits["tab_full"][0]
                yield "wait", "tab_full", index(e), parity(e), e["r"]
            yield from wait("P warps", "v_full", e, e["g"])
            if e["tail"]:
                yield from wait("P warps", "k_full", e, e["g"])
            for h in range(2):
                x = dict(e, h=h)
                yield from wait("P warps", "vt_empty", x, e["g"] - 1)
                yield from arrive("P warps", "vt_full", x)
            yield from arrive("P warps", "v_empty", e)
            if not state_only:
                yield from wait("P warps", "p_full", e, e["g"])
                yield from arrive("P warps", "p_ready", e)

    def state_warp():
        for e in chunks:
            yield from wait("state warps", "v_full", e, e["g"])
            for h in range(2):
                x = dict(e, h=h)
                yield from wait("state warps", "vt_empty", x, e["g"])
                yield from arrive("state warps", "vt_full", x)
            yield from arrive("state warps", "v_empty", e)
            if not state_only:
                yield from wait("state warps", "o_full", e, e["g"] - 1)
                yield from arrive("state warps", "s_full", e)
            yield from wait("state warps", "ds_full", e, e["g"])
            yield from arrive("state warps", "ds_empty", e)

    def out_warp():
        for e in chunks:
            yield from wait("output warps", "o_full", e, e["g"])
            yield from arrive("output warps", "o_empty", e)

    out = {"TMA": tma, "B": mma_b, **{f"P{i}": p_warp for i in range(4)}, **{f"S{i}": state_warp for i in range(4)}}
    if not state_only:
        out.update({"A": mma_a, "C": mma_c, **{f"O{i}": out_warp for i in range(4)}})
    return out


def run(init, roles, state_only, tails, held, at):
    """Steps all agents to the end, agent `held` standing still before its step `at` until nothing else moves; returns
    the agents that never finish."""
    m, live, steps = Machine(init, state_only), {}, {}
    for name, make in _agents(roles, state_only, tails).items():
        gen = make()
        live[name] = [gen, next(gen)]
        steps[name] = 0
    released = False
    while live:
        moved = False
        for name in list(live):
            if name == held and steps[name] >= at and not released:
                continue
            while name in live:
                gen, op = live[name]
                if op[0] == "wait":
                    if not m.done(op[1], op[2], op[3]):
                        break
                    assert op[4] in m.bar(op[1], op[2])[1], f"{name} passed {op[1]} before chunk {op[4]}"
                else:
                    m.arrive(*op[1:])
                steps[name] += 1
                moved = True
                try:
                    live[name][1] = next(gen)
                except StopIteration:
                    del live[name]
                if name == held and steps[name] >= at and not released:
                    break
        if not moved:
            if released or held is None:
                return {n: x[1] for n, x in live.items()}
            released = True
    return {}


@pytest.mark.parametrize("state_only,tails", [(0, False), (0, True), (1, False), (1, True)])
def test_every_role_may_be_late(kernel, state_only, tails):
    init, roles = kernel
    assert run(init, roles, state_only, tails, None, 0) == {}
    for name, make in _agents(roles, state_only, tails).items():
        if name[-1] in "123":
            continue  # (the warps of a role do the same)
        for at in range(sum(1 for _ in make())):
            stuck = run(init, roles, state_only, tails, name, at)
            assert stuck == {}, f"{name} held at its step {at}: {stuck}"
