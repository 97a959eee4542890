"""The marks of values that are not finite in tree attention, on the CPU under random delays.

The warpgroup that first meets an infinity or a NaN in a node's V takes it out of shared
memory and marks the stretch; every row that attends to the node gets it back when its
warpgroup is through with the stretch, if the mark is still there.  The marks are a ring.
Here the barrier model of the kernel runs with them: the last tile of every stretch holds
such a value, and a softmax thread may stall for long before it reads the mark.
"""
import os
import random
import re

import pytest

from test_tree_barriers import Model

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_cache_164_gb300", "csrc", "pkv_tree_attention.cu")


class Marked(Model):
    def __init__(self, seed, rows, slots, stretches, marks):
        super().__init__(seed, rows, slots, 1 if rows else 2, stretches)
        self.marks, self.clean = [0] * marks, set()

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
                if j == nt - 1:
                    slot, phase = self.place(True, place0, j, nt)
                    yield self.full[slot], phase
                    if (s, j) not in self.clean:  # marked, then taken out
                        self.marks[s % len(self.marks)] = s + 1
                        self.clean.add((s, j))
                if not self.rows and j == tiles[0] and s:
                    yield self.o_free, s - 1
                yield self.delay(0.3)
                self.arrive(self.p_ready[w][b])
                step += 1
            place0 += self.places(nt)
            if not self.rows and more:
                self.arrive(q_ready)
            yield self.pv_done[w][(step - 1) % 2], (step - 1) // 2
            if not self.rows:
                self.arrive(self.met)
                yield self.met, s
            yield self.delay(0.3) if self.r.random() < 0.8 else self.r.uniform(20, 200)
            if self.marks[s % len(self.marks)] != s + 1:
                self.fault = f"the mark of stretch {s} is gone"
            yield self.delay(0.3)
            if self.rows:
                if more:
                    self.arrive(q_ready)
            else:
                self.arrive(self.o_free)


def _faults(rows, slots, marks, seeds):
    found = []
    for seed in seeds:
        r = random.Random(seed)
        stretches = [2 * r.choice([1, 1, 1, 1, 2, 3]) for _ in range(r.randint(5, 14))]
        found.append(Marked(seed, rows, slots, stretches, marks).run())
    return [f for f in found if f]


@pytest.mark.parametrize("slots", [10, 16])
@pytest.mark.parametrize("rows", [False, True])
def test_no_mark_is_lost(rows, slots):
    with open(SOURCE) as f:
        marks = int(re.search(r"constexpr int kTreeMarks = (\d+);", f.read()).group(1))
    assert not _faults(rows, slots, marks, range(200))


def test_the_model_tells_a_ring_of_four_marks():
    assert any("is gone" in f for f in _faults(True, 16, 4, range(200)))
    assert not _faults(True, 10, 4, range(200))  # ten slots hold three stretches at most
