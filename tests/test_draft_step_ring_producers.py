"""The hand-off of the draft step's persistent kernel (csrc/draft_step.cu) with both of its producer warps,
modelled on the host. A barrier is what the hardware has: a count of arrivals and of bytes to come, a phase
that ends when both are nothing. One producer copies the state, the other the tokens and, with an arrival of
each of its lanes, the gates; both wait for an empty stage on their own, copies land in any order, each warp
of a group waits, meets the others and gives the stage back on its own. No stage may change while a group
reads it, each group must read its own items whole, and all must end. Stages, groups, barriers and arrivals
are read from the kernel's source."""
import os
import random
import re

import pytest

SOURCE = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_linear_attention_gb300",
                           "csrc", "draft_step.cu")).read()
RINGS = [tuple(map(int, m)) for m in re.findall(r"static_assert\(ring_is<StepSmem<\w+, \d+>>\((\d+), (\d+), (\d+)\)\)", SOURCE)]
FULL_ARRIVALS = sum(map(int, re.search(r"mbar_init\(&full\[s\], (\d+) \+ (\d+)\)", SOURCE).groups()))
WARPS = int(re.search(r"kGroupThreads = (\d+)", SOURCE).group(1)) // 32
assert "mbar_init(&empty[s], kGroupThreads / 32)" in SOURCE


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.bytes, self.phase = count, count, 0, 0

    def arrive(self, bytes=0):
        assert self.left > 0, "more arrivals than a phase takes"
        self.left -= 1
        self.bytes += bytes
        self._end()

    def land(self, bytes):
        self.bytes -= bytes
        self._end()

    def _end(self):
        if self.left == 0 and self.bytes == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        """What a wait for the end of the phase with this parity sees."""
        return self.phase % 2 != parity


def _run(stages, groups, fulls, items, rng, per_stage=False):
    fulls = stages if per_stage else fulls
    full, empty = [Barrier(FULL_ARRIVALS) for _ in range(fulls)], [Barrier(WARPS) for _ in range(stages)]
    held = [[None] * stages for _ in range(2)]       # item whose state, whose tokens a stage holds whole
    using = [0] * stages                             # warps that read a stage
    staged, flying = [0, 0], []                      # per producer; (producer, item, bytes or lanes, what)
    at = [[g] * WARPS for g in range(groups)]        # next item of each warp
    state = [["wait"] * WARPS for _ in range(groups)]
    done = 0
    while True:
        steps = []
        for p in range(2):
            k = staged[p]
            if k < items and empty[k % stages].passed((k // stages + 1) % 2):
                steps.append(("stage", p, 0))
        steps += [("land", i, 0) for i in range(len(flying))]
        for g in range(groups):
            for w in range(WARPS):
                k = at[g][w]
                if state[g][w] == "wait" and k < items and full[k % fulls].passed(k // fulls % 2):
                    steps.append(("arrive", g, w))
                elif state[g][w] == "read":
                    steps.append(("give back", g, w))
            if all(s == "here" for s in state[g]):   # the group's own barrier
                steps.append(("meet", g, 0))
        if not steps:
            return done == items and all(s == items for s in staged)
        what, i, w = rng.choice(steps)
        if what == "stage":
            k = staged[i]
            if using[k % stages]:
                return False                         # overwritten while it is read
            held[i][k % stages] = None
            staged[i] += 1
            full[k % fulls].arrive(8 if i == 0 else 4)
            flying += [(i, k, 4, "bytes")] * (2 if i == 0 else 1) + [(i, k, 32, "lanes")] * i
        elif what == "land":
            p, k, n, kind = flying.pop(i)
            if kind == "bytes":
                full[k % fulls].land(n)
            else:
                for _ in range(n):
                    full[k % fulls].arrive()
            if not any(f[:2] == (p, k) for f in flying):
                held[p][k % stages] = k
        elif what == "arrive":
            state[i][w] = "here"
        elif what == "meet":
            k = at[i][0]
            if any(held[p][k % stages] != k for p in range(2)):
                return False                         # another item's, or not all of it
            using[k % stages] += WARPS
            state[i] = ["read"] * WARPS
        else:
            k = at[i][w]
            using[k % stages] -= 1
            empty[k % stages].arrive()
            at[i][w], state[i][w] = k + groups, "wait"
            done += w == 0


def test_the_source_names_four_rings():
    assert len(RINGS) == 4 and FULL_ARRIVALS == 34 and WARPS == 4


@pytest.mark.parametrize("ring", sorted(set(RINGS)) + [(5, 3, 6), (7, 2, 8), (6, 4, 8)])
def test_every_group_reads_its_items_whole(ring):
    rng = random.Random(sum(ring))
    assert all(_run(*ring, 30, rng) for _ in range(60))


def test_a_full_barrier_per_stage_would_fail():
    rng = random.Random(3)

    def ok():
        try:
            return _run(6, 4, 6, 30, rng, per_stage=True)
        except AssertionError:
            return False
    assert not all(ok() for _ in range(100))
