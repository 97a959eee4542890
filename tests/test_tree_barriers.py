"""The barrier protocol of the tree-attention kernel, on the CPU under random delays.

tree_attention_kernel's roles (four producers, two product issuers, two softmax
warpgroups) meet at mbarriers, and every wait names a phase by its parity alone:
a wait for phase f also passes when phase f - 2 is the last complete one.  This
discrete-event model runs the roles' waits and arrivals as the kernel orders
them, with random delays, and checks that no wait passes before the phase it
means, that every product reads the tile it means, and that nothing deadlocks.
The last test shows that the model tells a faulty form: one ring of slots walked
by two issuers that take every other tile.
"""
import heapq
import random

import pytest


class Barrier:
    def __init__(self, name, count):
        self.name, self.count = name, count
        self.pending = self.done = 0
        self.waiting = []


class Model:
    def __init__(self, seed, rows, slots, rings, stretches):
        self.r = random.Random(seed)
        self.now, self.order, self.events, self.fault = 0.0, 0, [], None
        self.rows, self.slots, self.rings, self.stretches = rows, slots, rings, stretches
        self.full = [Barrier(f"full{i}", 1) for i in range(slots)]
        # a tile's readers: both issuers, or the one that owns the tile
        self.empty = [Barrier(f"empty{i}", 2 if rows else 1) for i in range(slots)]
        pair = lambda name, n: [[Barrier(f"{name}{w}{b}", n) for b in range(2)]  # noqa: E731
                                for w in range(2)]
        self.s_full, self.p_ready, self.pv_done = pair("s", 1), pair("p", 2), pair("pv", 1)
        self.q_ready = [Barrier("q0", 2 if rows else 4), Barrier("q1", 2)]
        self.met, self.o_free = Barrier("met", 4), Barrier("o_free", 4)
        self.holds = [None] * slots

    # -- events ---------------------------------------------------------------
    def later(self, delay, f):
        self.order += 1
        heapq.heappush(self.events, (self.now + delay, self.order, f))

    def arrive(self, bar):
        bar.pending += 1
        if bar.pending == bar.count:
            bar.pending, bar.done = 0, bar.done + 1
            waiting, bar.waiting = bar.waiting, []
            for role, phase in waiting:
                self.wait(role, bar, phase)

    def wait(self, role, bar, phase):
        if (bar.done - 1) % 2 == phase % 2:  # by parity; a fresh barrier passes parity 1
            if bar.done <= phase:
                self.fault = f"{bar.name}: a wait for phase {phase} passed after {bar.done}"
            self.later(0, lambda: self.step(role))
        else:
            bar.waiting.append((role, phase))

    def step(self, role):
        try:
            what = next(role)
        except StopIteration:
            self.alive -= 1
            return
        if isinstance(what, float):
            self.later(what, lambda: self.step(role))
        else:
            self.wait(role, *what)

    def run(self):
        roles = [self.producer(v, odd) for v in (False, True) for odd in (0, 1)]
        roles += [self.issuer(w) for w in (0, 1)]
        roles += [self.softmax(w) for w in (0, 0, 1, 1)]  # two threads a warpgroup
        self.alive = len(roles)
        for role in roles:
            self.later(self.r.random(), lambda role=role: self.step(role))
        while self.events and not self.fault:
            self.now, _, f = heapq.heappop(self.events)
            f()
        return self.fault or ("deadlock" if self.alive else None)

    def delay(self, mean):  # mostly near the mean, sometimes far above it
        if self.r.random() < 0.9:
            return self.r.expovariate(1 / mean)
        return mean * self.r.uniform(3, 30)

    # -- the ring of slots ------------------------------------------------------
    def place(self, is_v, place0, j, nt):
        """(slot, phase) of tile j of a stretch of nt tiles."""
        two = self.rings == 2 and not self.rows
        size = self.slots // 2 if two else self.slots
        k, n = (j >> 1, nt >> 1) if two else (j, nt)
        ahead = 4 if self.rings == 1 and not self.rows else 2
        at = place0 + (min(k + ahead, n) + k if is_v else k if k < ahead else 2 * k - ahead + 1)
        return at % size + (j % 2 * size if two else 0), at // size

    def places(self, nt):
        return nt if self.rings == 2 and not self.rows else 2 * nt

    # -- roles ------------------------------------------------------------------
    def producer(self, is_v, odd):
        place0 = 0
        for s, nt in enumerate(self.stretches):
            for j in range(odd, nt, 2):
                slot, phase = self.place(is_v, place0, j, nt)
                if phase:
                    yield self.empty[slot], phase - 1
                yield self.delay(0.1)

                def land(slot=slot, tile=(s, is_v, j)):
                    self.holds[slot] = tile
                    self.arrive(self.full[slot])
                self.later(self.delay(1.0), land)
            place0 += self.places(nt)

    def issuer(self, w):
        place0 = steps0 = 0
        last = [0.0]  # the tensor core completes an issuer's products in order

        def product(bars):
            last[0] = max(last[0], self.now) + self.r.uniform(0.2, 0.6)
            for bar in bars:
                self.later(last[0] - self.now, lambda bar=bar: self.arrive(bar))

        for s, nt in enumerate(self.stretches):
            steps = nt if self.rows else nt // 2

            def one(is_v, k):
                j = k if self.rows else 2 * k + w
                slot, phase = self.place(is_v, place0, j, nt)
                b = (steps0 + k) % 2
                yield self.full[slot], phase
                if self.holds[slot] != (s, is_v, j):
                    self.fault = f"a product of {(s, is_v, j)} reads {self.holds[slot]}"
                if is_v:
                    yield self.p_ready[w][b], (steps0 + k) // 2
                product([(self.pv_done if is_v else self.s_full)[w][b], self.empty[slot]])

            yield self.q_ready[w if self.rows else 0], s
            for k in range(min(2, steps)):
                yield from one(False, k)
            for k in range(steps):
                yield from one(True, k)
                yield self.delay(0.05)
                if k + 2 < steps:
                    yield from one(False, k + 2)
            place0 += self.places(nt)
            steps0 += steps

    def softmax(self, w):
        place0 = step = 0
        q_ready = self.q_ready[w if self.rows else 0]
        self.arrive(q_ready)
        for s, nt in enumerate(self.stretches):
            more = s + 1 < len(self.stretches)
            tiles = range(nt) if self.rows else range(w, nt, 2)
            for j in tiles:
                b = step % 2
                yield self.s_full[w][b], step // 2
                if self.r.random() < 0.3:  # a masked tile: V is looked through
                    slot, phase = self.place(True, place0, j, nt)
                    yield self.full[slot], phase
                    if self.holds[slot] != (s, True, j):
                        self.fault = f"V {(s, j)} looked for in {self.holds[slot]}"
                if not self.rows and j == tiles[0] and s:
                    yield self.o_free, s - 1
                yield self.delay(0.7)
                if j != tiles[0] and self.r.random() < 0.2:  # O is rescaled
                    yield self.pv_done[w][1 - b], (step - 1) // 2
                self.arrive(self.p_ready[w][b])
                step += 1
            place0 += self.places(nt)
            if not self.rows and more:
                self.arrive(q_ready)
            yield self.pv_done[w][(step - 1) % 2], (step - 1) // 2
            if not self.rows:
                self.arrive(self.met)
                yield self.met, s
            yield self.delay(0.5)
            if self.rows:
                if more:
                    self.arrive(q_ready)
            else:
                self.arrive(self.o_free)


def _faults(rows, slots, rings, seeds):
    found = []
    for seed in seeds:
        r = random.Random(seed)
        stretches = [2 * r.choice([1, 1, 2, 3, 5, 12, 30]) for _ in range(r.randint(1, 7))]
        found.append(Model(seed, rows, slots, rings, stretches).run())
    return [f for f in found if f]


@pytest.mark.parametrize("slots", [10, 16])
@pytest.mark.parametrize("rows", [False, True])
def test_no_wait_passes_early_and_nothing_deadlocks(rows, slots):
    assert not _faults(rows, slots, 1 if rows else 2, range(150))


def test_the_model_tells_one_ring_for_two_issuers():
    found = _faults(False, 10, 1, range(60))
    assert any("passed after" in f for f in found)
