"""The order of the chunk kernel of the gated delta rule (csrc/delta_chunk.cuh), checked on the CPU: its roles' reads and writes of shared
memory and TMEM, its barriers and its products as a graph of what must come before what, for one sequence of several chunks, for blocks that go on
from one sequence to the next, for each I/O type and head size, with and without outputs and new states.

* Two accesses that overlap, one of them a write, are joined by a path.
* An arrival on a phase of a barrier comes after the phase before has ended, and a wait for a phase before the next one has ended: the parity that a
  wait looks at tells two neighbouring phases apart, no more, and a wait that is overtaken runs out.

`test_the_graph_is_that_of_the_source` holds the graph to the source: the waits, arrivals and commits of each role in their order, and where things
lie in TMEM.
"""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "bit_gated_delta_gb300", "csrc", "delta_chunk.cuh")
W, P_, D2, D4, D0 = 256, 320, 384, 384, 448


class Shape:
    def __init__(self, d, f32):
        self.d, self.f32 = d, f32
        self.NB, self.NV = (3 if not f32 else 2 if d == 64 else 1), (1 if f32 and d == 128 else 2)
        self.NM, self.NO, self.NQ, self.D3 = (1, 3, 3, 64) if f32 else (2, 2, 2, 0)
        self.NS = 3

    def a1(self, part):
        return 64 * part

    def a2(self, part):
        return 128 + 32 * part

    def a3(self, part):
        return 32 * part if self.f32 and part < 2 else 128 + 32 * part

    def a4(self, part):
        return W + 32 * part if part < 2 else 224


class Graph:
    """Nodes in program order of their actor; `pipe` is the tensor core, whose products run in the order of their issue."""

    def __init__(self):
        self.after, self.access, self.last = [], [], {}
        self.arrivals, self.waits, self.meetings = {}, [], {}

    def node(self, actor, extra=()):
        n = len(self.after)
        self.after.append(set(extra) | ({self.last[actor]} if actor in self.last else set()))
        self.last[actor] = n
        return n

    def touch(self, actor, what, where, first=0, last=1):
        n = self.node(actor)
        self.access.append((n, what == "w", where, first, last))

    def product(self, reads, writes):
        n = self.node("pipe", {self.last["mma"]} if "mma" in self.last else ())
        for what, list_ in (("r", reads), ("w", writes)):
            self.access.extend((n, what == "w", *x) for x in list_)

    def arrive(self, actor, bar):
        self.arrivals.setdefault(bar, {}).setdefault(actor, []).append(self.node(actor))

    def commit(self, bar):
        self.arrivals.setdefault(bar, {}).setdefault("pipe", []).append(self.node("pipe", {self.last["mma"]} if "mma" in self.last else ()))

    def wait(self, actor, bar, phase):
        self.waits.append((self.node(actor), bar, phase))

    def meet(self, actor, name):
        """A named barrier: turns of all its actors join."""
        self.meetings.setdefault(name, {}).setdefault(actor, []).append((self.node(actor), self.node(actor)))

    def close(self):
        for turns in self.meetings.values():
            for joined in zip(*turns.values()):
                for _, out in joined:
                    self.after[out] |= {i for i, _ in joined}
        for n, bar, phase in self.waits:
            for own in self.arrivals[bar].values():
                self.after[n].add(own[phase])
        # what comes before each node, as bits (in an order in which every node comes after those before it)
        self.before, done = [0] * len(self.after), [False] * len(self.after)
        stack = list(range(len(self.after)))
        while stack:
            n = stack[-1]
            todo = [m for m in self.after[n] if not done[m]]
            if done[n] or not todo:
                stack.pop()
                if not done[n]:
                    for m in self.after[n]:
                        self.before[n] |= self.before[m] | 1 << m
                    done[n] = True
            else:
                assert len(stack) < 10 * len(self.after), "a wait for something that comes after it"
                stack.extend(todo)

    def comes_before(self, a, b):
        return a == b or self.before[b] >> a & 1

    def faults(self):
        self.close()
        found = set()
        by = {}
        for x in self.access:
            by.setdefault(x[2], []).append(x)
        for where, list_ in by.items():
            for i, (n, w, _, f, l) in enumerate(list_):
                for m, w2, _, f2, l2 in list_[:i]:
                    if (w or w2) and f < l2 and f2 < l and not self.comes_before(n, m) and not self.comes_before(m, n):
                        found.add((where, max(f, f2), min(l, l2)))
        for bar, own in self.arrivals.items():
            for actor, at in own.items():
                for other in own.values():
                    assert len(other) == len(at), bar
                    found |= {("arrival", bar) for i in range(1, len(at)) if not self.comes_before(other[i - 1], at[i])}
        for n, bar, phase in self.waits:
            own = self.arrivals[bar]
            if len(next(iter(own.values()))) > phase + 1 and not any(self.comes_before(n, at[phase + 1]) for at in own.values()):
                found.add(("overtaken", bar))
        return found


def kernel(d, f32, out, write, units, waits_for_reads=True, ready_by_buffer=True):
    """The graph of a block that goes through units of so many chunks of 64 tokens each."""
    z, g_ = Shape(d, f32), Graph()
    tm = "tmem"
    o_ready = (lambda g: (f"o_ready{g % z.NV}", g // z.NV)) if ready_by_buffer else (lambda g: ("o_ready", g))

    def columns(j):
        me, half, t0, held, g = f"columns{j}", j >> 1, 16 * j, z.d // 4, 0

        def store():
            g_.touch(me, "w", f"v{(g - 1) % z.NV}", t0, t0 + 16)
            g_.arrive(me, o_ready(g - 1)[0])
        for chunks in units:
            for c in range(chunks + 1):
                if c > 0 and write:
                    g_.wait(me, "s_done", g - 1)
                    g_.touch(me, "r", tm, z.D3 + j * held, z.D3 + (j + 1) * held)
                    g_.meet(me, "quarter")
                if c < chunks:
                    for k in range(z.NS):
                        g_.touch(me, "w", tm, z.a1(k) + j * held // 2, z.a1(k) + (j + 1) * held // 2)
                    g_.arrive(me, "a1")
                if out and c > 0:
                    g_.wait(me, "o_done", g - 1)
                    g_.touch(me, "r", tm, D4 + t0, D4 + t0 + 16)
                    g_.touch(me, "r", tm, P_ + t0, P_ + t0 + 16)
                    g_.touch(me, "r", f"G{(g - 1) % 3}")
                    g_.arrive(me, "o_read")
                    if z.NV == 1:
                        store()
                if c < chunks:
                    g_.wait(me, f"ready{g % 3}", g // 3)
                    g_.wait(me, "w_done", g)
                    if f32 and out:
                        g_.wait(me, "p_done", g)
                    g_.touch(me, "r", f"v{g % z.NV}", t0, t0 + 16)
                    g_.touch(me, "r", tm, W + t0, W + t0 + 16)
                    g_.touch(me, "r", f"G{g % 3}")
                    g_.touch(me, "r", f"gates{g % 3}")
                    for k in range(3):
                        g_.touch(me, "w", tm, z.a2(k) + t0 // 2, z.a2(k) + t0 // 2 + 8)
                    g_.arrive(me, f"a2{half}")
                if z.NV > 1 and out and c > 0:
                    store()
                if c == chunks:
                    break
                g_.touch(me, "r", f"G{g % 3}")
                g_.wait(me, f"u_done{half}", g)
                if write:
                    g_.touch(me, "r", tm, D2 + t0, D2 + t0 + 16)
                    g_.touch(me, "r", f"rho{g % 3}")
                    for k in range(3):
                        g_.touch(me, "w", tm, z.a3(k) + t0 // 2, z.a3(k) + t0 // 2 + 8)
                    g_.arrive(me, f"a3{half}")
                if out:
                    if half == 0:
                        g_.wait(me, "u_done1", g)
                    g_.touch(me, "r", tm, D2 + t0, D2 + t0 + 16)
                    for k in range(z.NO):
                        g_.touch(me, "w", tm, z.a4(k) + t0 // 2, z.a4(k) + t0 // 2 + 8)
                    g_.arrive(me, "a4")
                g += 1

    n = sum(units)

    def rows_in(me, g, first, last):
        if g >= z.NB:
            g_.wait(me, f"x_free{g % z.NB}", g // z.NB - 1)
        for x in ("k", "q")[:1 + out]:
            g_.touch(me, "w", f"{x}{g % z.NB}", first, last)
        g_.arrive(me, f"x_full{g % z.NB}")

    def tables(isq):
        me = f"tables{isq}"
        for g in range(n):
            if f32:
                rows_in(me, g, isq, isq + 1)
            if not isq:
                g_.touch(me, "w", f"gates{g % 3}")
            g_.meet(me, "tables")
            if g >= z.NM:
                g_.wait(me, f"m_free{g % z.NM}", g // z.NM - 1)
            g_.wait(me, "g_done", g)
            g_.touch(me, "r", tm, D0, D0 + 64)
            g_.touch(me, "r", f"gates{g % 3}")
            if isq:
                g_.touch(me, "w", f"rho{g % 3}")
                if out:
                    g_.touch(me, "w", f"P{g & 1}")
                g_.touch(me, "w", f"G{g % 3}")
            else:
                g_.touch(me, "w", f"M{g % z.NM}")
            g_.arrive(me, f"ready{g % 3}")
            g_.arrive(me, f"m_ready{g % z.NM}")

    def inverses():
        me = "inverses"
        for g in range(n):
            g_.wait(me, f"m_ready{g % z.NM}", g // z.NM)
            g_.touch(me, "w", f"M{g % z.NM}")
            if g:
                g_.wait(me, "u_done1", g - 1)
            g_.touch(me, "w", "T")
            g_.arrive(me, "t_ready")
            g_.arrive(me, f"m_free{g % z.NM}")

    def copies():
        for g in range(n):
            if not f32:
                rows_in("rows", g, 0, 2)
            if g >= z.NV:
                if out:
                    g_.wait("v", f"o_free{g % z.NV}", g // z.NV - 1)
                else:
                    g_.wait("v", f"x_free{(g - z.NV) % z.NB}", (g - z.NV) // z.NB)
            g_.touch("v", "w", f"v{g % z.NV}", 0, 64)
            g_.arrive("v", f"ready{g % 3}")
            if out:
                g_.wait("o", *o_ready(g))
                g_.touch("o", "r", f"v{g % z.NV}", 0, 64)
                g_.arrive("o", f"o_free{g % z.NV}")

    def products():
        me, part = "mma", lambda at, count, first, last: [(tm, at(k) + first, at(k) + last) for k in range(count)]

        def dots(g):
            g_.wait(me, f"x_full{g % z.NB}", g // z.NB)
            g_.product([(f"{x}{g % z.NB}", 0, 2) for x in ("k", "q")[:1 + out]], [(tm, D0, D0 + 64)])
            g_.commit("g_done")
        dots(0)
        for g in range(n):
            def of_q():
                if g:
                    g_.wait(me, "o_read", g - 1)
                g_.product(part(z.a1, z.NQ, 0, d // 2) + [(f"q{g % z.NB}", 0, 2)], [(tm, P_, P_ + 64)])
                if f32:
                    g_.commit("p_done")
            g_.wait(me, "a1", g)
            g_.product(part(z.a1, z.NS, 0, d // 2) + [(f"k{g % z.NB}", 0, 2)], [(tm, W, W + 64)])
            g_.commit("w_done")
            if f32 and out:
                of_q()
            if z.NB > 1 and g + 1 < n:
                g_.wait(me, f"ready{g % 3}", g // 3)
                dots(g + 1)
            g_.wait(me, "t_ready", g)
            if waits_for_reads and not f32 and out and g:
                g_.wait(me, "o_read", g - 1)
            for r in range(2):
                g_.wait(me, f"a2{r}", g)
                g_.product(part(z.a2, 3, 16 * r, 16 * r + 16) + [("T", 0, 1)], [(tm, D2 + 32 * r, D2 + 64)])
                g_.commit(f"u_done{r}")
            if not f32 and out:
                of_q()
            if write:
                for r in range(2):
                    g_.wait(me, f"a3{r}", g)
                    g_.product(part(z.a3, 3, 16 * r, 16 * r + 16) + [(f"k{g % z.NB}", 0, 2)], [(tm, z.D3, z.D3 + d)])
                g_.commit("s_done")
            g_.commit(f"x_free{g % z.NB}")
            if out:
                g_.wait(me, "a4", g)
                g_.product(part(z.a4, z.NO, 0, 32) + [(f"P{g & 1}", 0, 1)], [(tm, D4, D4 + 64)])
                g_.commit("o_done")
            if z.NB == 1 and g + 1 < n:
                dots(g + 1)

    for j in range(4):
        columns(j)
    tables(0), tables(1), inverses(), copies(), products()
    return g_


CALLS = [(True, True), (False, True), (True, False)]     # outputs and states (chunk), states only (keep), outputs only (draft)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out,write", CALLS)
def test_every_access_has_its_place(d, f32, out, write):
    for units in ([1] * 7,) + (([7], [3, 1, 2, 1]) if write else ()):
        assert kernel(d, f32, out, write, units).faults() == set()


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_are_read_before_u_is_written_over_them(d):
    """Without the wait for o_read before the products of u, those of the first half of the tokens may write over the outputs of the second."""
    for units in ([4], [3, 1, 2, 1]):
        assert kernel(d, False, True, True, units, waits_for_reads=False).faults() == {("tmem", D4 + 32, D4 + 48), ("tmem", D4 + 48, D4 + 64)}


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_are_announced_by_buffer(d, f32):
    """With one barrier for both buffers of outputs the columns' warps may announce chunk g + 1 (into the buffer that g - 1 has left) before the warp
    that copies outputs has looked for chunk g; it would wait for g + 2, which waits for it."""
    for units in ([4], [3, 1, 2, 1]):
        found = kernel(d, f32, True, True, units, ready_by_buffer=False).faults()
        assert found == (set() if Shape(d, f32).NV == 1 else {("overtaken", "o_ready")})


def test_the_graph_is_that_of_the_source():
    text = re.sub(r"//[^\n]*", lambda m: m.group() if "-----" in m.group() else "", open(SOURCE).read())
    assert "W = 256, P = 320, D2 = 384, D4 = 384, D0 = 448, D3 = F32 ? 64 : 0;" in text
    assert "a1(int part) { return 64 * part; }" in text and "a2(int part) { return 128 + 32 * part; }" in text
    assert "a3(int part) { return F32 && part < 2 ? 32 * part : 128 + 32 * part; }" in text
    assert "a4(int part) { return part < 2 ? W + 32 * part : 224; }" in text
    for x in ("NO = F32 ? 3 : 2;", "NB = !F32 ? 3 : D == 64 ? 2 : 1, NV = F32 && D == 128 ? 1 : 2;", "NM = F32 ? 1 : 2;", "NS = 3, NQ = F32 ? 3 : 2;"):
        assert x in text
    roles = re.split(r"//\s*-{20,}[^\n]*", text)[1:]
    assert len(roles) == 5
    calls = re.compile(r"\b(wait|arrive|commit)\(([^;,]*)(?:, ([^;]*))?\);|(bar\.sync) %0|\b(sync4<\d>)\(\)")
    got = [[" ".join(filter(None, m.groups())) for m in calls.finditer(r)] for r in roles]
    columns = ["wait o_done g - 1", "arrive o_read", "arrive &o_ready[(g - 1) % NV]", "wait s_done g - 1", "bar.sync", "arrive a1", "wait &ready[g3()] r3()", "wait w_done g",
               "wait p_done g", "arrive a2 + half", "wait u_done + half g", "arrive a3 + half", "wait u_done + 1 g", "arrive a4"]
    tables = ["wait &x_free[at_x()] round_x() - 1", "arrive &x_full[at_x()]", "sync4<1>", "wait &m_free[g % NM] g / NM - 1", "wait g_done g",
              "arrive &ready[g3()]", "arrive &m_ready[g % NM]"]
    inverses = ["wait &m_ready[g % NM] g / NM"] + ["sync4<6>"] * 5 + ["wait u_done + 1 g - 1", "arrive t_ready", "arrive &m_free[g % NM]"]
    copies = ["wait &x_free[at_x()] round_x() - 1", "wait &o_free[g % NV] g / NV - 1", "wait &x_free[(g - NV) % NB] (g - NV) / NB",
              "arrive what == 0 ? &x_full[at_x()] : &ready[g3()]", "wait &o_ready[g % NV] g / NV", "arrive &o_free[g % NV]"]
    products = ["wait &x_full[at_x()] round_x()", "commit g_done", "wait drain 0", "wait a1 now", "commit w_done", "wait o_read now - 1", "commit p_done",
                "wait &ready[g3()] r3()", "wait t_ready now", "wait o_read now - 1", "wait a2 + r now", "commit u_done + r", "wait a3 + r now",
                "commit s_done", "commit &x_free[buf]", "wait a4 now", "commit o_done", "commit drain"]
    assert got == [columns, tables, inverses, copies, products]
