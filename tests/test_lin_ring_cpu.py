"""The barriers of the bf16 linear-attention kernel (csrc/kda_lin_tc.cu) as a
model: its warps as generators that wait on mbarriers by parity, its loads and
products as events that end in any order the hardware allows, run under random
schedules.  What is looked for: a tile read that is not (or no longer) in its
slot, a load over a tile that somebody still has to read, anything in flight
when all warps have ended, and standstill.

The roles, waits and arrivals are those of the kernel, line by line; a chunk is
its number of 32-token quarters and whether its last one is cut short.
"""
import random

import pytest

V_BARS = 4  # kVBars


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        assert self.pending >= 0, "an arrival too many in one phase"
        self.check()

    def landed(self):
        self.tx -= 1
        self.check()

    def check(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def passes(self, parity):  # true when the phase of that parity is not the current one
        return (self.phase & 1) != parity


class Ring:
    """One CTA.  kind: fwd (R W V a chunk), sum (W V) or dq (E R W V).  chunks:
    (quarters, short) in the order of the pass.  v_by_slot: V on its slot's
    barrier, without v_seen, to see that the model finds what that allows."""

    def __init__(self, kind, slots, chunks, rng, v_by_slot=False):
        self.kind, self.slots, self.chunks, self.rng, self.by_slot = kind, slots, chunks, rng, v_by_slot
        self.names = {"fwd": "RWV", "sum": "WV", "dq": "ERWV"}[kind]
        self.tiles = len(self.names)
        self.groups = 4 if kind == "sum" else 2
        self.out = kind != "sum"
        bars = lambda n, count: [Bar(count) for _ in range(n)]  # noqa: E731
        self.full, self.free = bars(slots, 1), bars(slots, 2)
        self.v_full, self.v_seen = bars(V_BARS, 1), bars(V_BARS, 2 * self.groups)  # two warps stand for a group's four
        self.a_full, self.p_full, self.a_free = bars(2, 1), bars(2, 1), bars(2, 1)
        self.vb_full, self.vb_free = bars(self.groups, 2), bars(self.groups, 1)
        self.s_full, self.kv_done, self.qs_done, self.o_scaled, self.pv_done, self.o_free = bars(6, 1)
        self.clean = bars(2, 2)
        self.content = [None] * slots      # (chunk, tile name) that has landed
        self.readers = [0] * slots         # of the tile in the slot: still to come
        self.buffer = [None] * self.groups  # (chunk, quarter) converted, per warp
        self.loads = []
        self.pipes = {21: [], 22: []}      # issued products and commits, in order
        self.zeroed = set()

    # ---- addresses
    def index(self, c, name):
        return c * self.tiles + self.names.index(name)

    def slot(self, c, name):
        return self.index(c, name) % self.slots

    def phase(self, c, name):
        return self.index(c, name) // self.slots & 1

    def read(self, c, name):
        assert self.content[self.slot(c, name)] == (c, name), f"{name}{c} read, slot holds {self.content[self.slot(c, name)]}"

    def wait_full(self, c, name):
        return self.full[self.slot(c, name)], self.phase(c, name)

    def wait_v(self, c):
        if self.by_slot:
            return self.wait_full(c, "V")
        return self.v_full[c % V_BARS], c // V_BARS & 1

    # ---- roles
    def tma(self):
        for c in range(len(self.chunks)):
            for name in self.names:
                s, x = self.slot(c, name), self.index(c, name)
                if x >= self.slots:
                    yield self.free[s], self.phase(c, name) ^ 1
                if name == "V" and not self.by_slot and c >= V_BARS:
                    yield self.v_seen[c % V_BARS], (c // V_BARS - 1) & 1
                assert self.readers[s] == 0, f"{name}{c} loaded over {self.content[s]}, still to be read"
                self.content[s] = None
                bar = self.v_full[c % V_BARS] if name == "V" and not self.by_slot else self.full[s]
                bar.arrive(tx=1)
                if bar is not self.full[s]:
                    self.full[s].arrive()
                self.readers[s] = 2 * self.chunks[c][0] if name == "V" else 0  # reads by the V groups
                self.loads.append((bar, s, (c, name)))
        for x in range(max(0, len(self.chunks) * self.tiles - self.slots), len(self.chunks) * self.tiles):
            yield self.free[x % self.slots], x // self.slots & 1

    def v_warp(self, grp, w):
        quarters = 0
        for c, (nq, short) in enumerate(self.chunks):
            yield self.wait_v(c)
            if not self.by_slot:
                self.v_seen[c % V_BARS].arrive()
            if short and (quarters + nq - 1) % self.groups == grp:
                yield self.wait_full(c, "W")
                self.read(c, "W")
                self.read(c, "V")
                self.zeroed.add((c, w))
                self.clean[c & 1].arrive()
            for q in range(nq):
                if quarters % self.groups == grp:
                    if quarters >= self.groups:
                        yield self.vb_free[grp], (quarters // self.groups - 1) & 1
                    self.read(c, "V")
                    self.readers[self.slot(c, "V")] -= 1
                    self.buffer[grp] = (c, q)
                    self.vb_full[grp].arrive()
                quarters += 1

    def p_role(self):
        for c in range(len(self.chunks)):
            ab, use = (0, c) if self.kind == "dq" else (c & 1, c >> 1)
            yield self.a_full[ab], use & 1
            self.p_full[ab].arrive()

    def s_role(self):
        for c in range(len(self.chunks) + 1):  # (the last time for the state behind the segment)
            if c > 0:
                yield self.kv_done, (c - 1) & 1
                if self.out:
                    yield self.qs_done, (c - 1) & 1
            if c < len(self.chunks):
                self.s_full.arrive()

    def o_role(self):
        for c in range(len(self.chunks)):
            yield self.qs_done, c & 1
            self.o_scaled.arrive()
            yield self.pv_done, c & 1
            self.o_free.arrive()

    def product(self, pipe, c, names, buffer=None):
        self.pipes[pipe].append((c, names, buffer))

    def commit(self, pipe, *bars):
        self.pipes[pipe] += bars

    def release(self, pipe, c, name):
        self.commit(pipe, self.free[self.slot(c, name)])

    def mma_state(self):
        n, quarters, k, cleans, dq = len(self.chunks), 0, 0, [0, 0], self.kind == "dq"

        def begin():
            nonlocal k
            if k >= n:
                return
            for name in ("R" if self.out else "") + "W" + ("E" if dq else ""):
                yield self.wait_full(k, name)
            if dq:
                yield self.wait_v(k)
            if self.chunks[k][1]:
                yield self.clean[k & 1], cleans[k & 1] & 1
                cleans[k & 1] += 1
            if self.out:
                ab, use = (0, k) if dq else (k & 1, k >> 1)
                if use:
                    yield self.a_free[ab], (use - 1) & 1
                self.product(21, k, "RW")
                if dq:
                    self.product(21, k, "EV")
                    self.release(21, k, "E")
                    self.release(21, k, "E")
                self.commit(21, self.a_full[ab])
                self.release(21, k, "R")
            k += 1

        if not dq:
            yield from begin()
        for c, (nq, _) in enumerate(self.chunks):
            if dq:
                yield from begin()
            yield self.s_full, c & 1
            for q in range(nq):
                if q == min(nq, 2) and not dq:
                    yield from begin()
                vb = quarters % self.groups
                yield self.vb_full[vb], quarters // self.groups & 1
                self.product(21, c, "W", (vb, q))
                self.commit(21, self.vb_free[vb])
                if q == nq - 1:
                    self.commit(21, self.kv_done)
                    for name in "WWV" + ("" if self.out else "V"):
                        self.release(21, c, name)
                quarters += 1
            if nq <= 2 and not dq:
                yield from begin()

    def mma_out(self):
        cleans, dq = [0, 0], self.kind == "dq"
        for c, (nq, short) in enumerate(self.chunks):
            if short:
                yield self.clean[c & 1], cleans[c & 1] & 1
                cleans[c & 1] += 1
            yield self.wait_full(c, "R")
            yield self.s_full, c & 1
            if c > 0:
                yield self.o_free, (c - 1) & 1
            self.product(22, c, "R")
            self.commit(22, self.qs_done)
            self.release(22, c, "R")
            ab, use = (0, c) if dq else (c & 1, c >> 1)
            yield self.wait_v(c)
            yield self.p_full[ab], use & 1
            yield self.o_scaled, c & 1
            self.product(22, c, "V")
            self.commit(22, self.pv_done, self.a_free[ab])
            self.release(22, c, "V")

    # ---- events
    def land(self):
        bar, s, what = self.loads.pop(self.rng.randrange(len(self.loads)))  # in any order
        self.content[s] = what
        bar.landed()

    def step_pipe(self, pipe):
        op = self.pipes[pipe].pop(0)
        if isinstance(op, Bar):
            op.arrive()
            return
        c, names, buffer = op
        for name in names:
            self.read(c, name)
        if self.chunks[c][1] and set(names) & set("WV"):
            assert (c, 0) in self.zeroed and (c, 1) in self.zeroed, "a short chunk's rows are not cleared"
        if buffer:
            assert self.buffer[buffer[0]] == (c, buffer[1])

    def run(self):
        roles = [self.tma(), self.s_role(), self.mma_state()] + [self.v_warp(g, w) for g in range(self.groups) for w in (0, 1)]
        if self.out:
            roles += [self.p_role(), self.o_role(), self.mma_out()]
        waits = {i: next(r, None) for i, r in enumerate(roles)}
        speed = {i: self.rng.choice((1, 1, 8, 64)) for i in waits}
        slow_loads = self.rng.choice((1, 8, 64, 400))
        while True:
            ready = [(i, speed[i]) for i, w in waits.items() if w is not None and w[0].passes(w[1])]
            ready += [("land", 64 / slow_loads)] * bool(self.loads)
            ready += [(p, 8) for p in self.pipes if self.pipes[p]]
            if not ready:
                break
            who = self.rng.choices([r[0] for r in ready], [r[1] for r in ready])[0]
            if who == "land":
                self.land()
            elif who in self.pipes:
                self.step_pipe(who)
            else:
                waits[who] = next(roles[who], None)
            if not any(waits.values()):  # every warp is at the CTA's end
                assert not self.loads and not any(self.pipes.values()), "in flight behind the CTA's end"
        assert all(w is None for w in waits.values()), f"standstill: {[i for i, w in waits.items() if w is not None]}"


def chunk_list(kind, rng):
    n = rng.randint(1, 14)
    if kind == "sum":  # one sequence: the short chunk is its last, or the first of a reversed pass
        out = [(4, False)] * n
        if rng.random() < 0.8:
            out[rng.choice((0, -1))] = (rng.randint(1, 4), True)
        return out
    tail = rng.choice((1, 1, 2, 4))
    return [(4, False) if rng.random() < 0.4 else (rng.randint(1, tail), rng.random() < 0.9) for _ in range(n)]


@pytest.mark.parametrize("kind,slots", [("fwd", 5), ("fwd", 6), ("fwd", 7), ("fwd", 8), ("sum", 4),
                                        ("sum", 5), ("sum", 6), ("sum", 7), ("sum", 8), ("dq", 5), ("dq", 6), ("dq", 7), ("dq", 8)])
def test_every_schedule_reads_what_it_waited_for(kind, slots):
    for seed in range(200):
        rng = random.Random(f"{kind} {slots} {seed}")
        Ring(kind, slots, chunk_list(kind, rng), rng).run()


@pytest.mark.parametrize("kind,slots", [("fwd", 5), ("fwd", 8), ("dq", 5), ("sum", 5)])
def test_the_model_finds_waits_on_a_slot_that_miss_its_phases(kind, slots):
    found = 0
    for seed in range(200):
        rng = random.Random(f"{kind} {slots} {seed}")
        try:
            Ring(kind, slots, chunk_list(kind, rng), rng, v_by_slot=True).run()
        except AssertionError:
            found += 1
    assert found
