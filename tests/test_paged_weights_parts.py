"""How the four groups of the accumulated weights' kernel (csrc/paged_weights.cu) hand partial sums to one another, modelled on
the host: score tiles go to the groups in turn, tile by tile in order as far as their buffers are free; the group with an
item's first tile collects the others' sums, each of which lies in one slot of its sender. Groups run at any speed and
every wait looks at a barrier's parity as the kernel's do. Each sum must be the item's own, and all must end."""
import os
import random
import re

import pytest

from gated_linear_attention_gb300 import build

GROUPS = 4


def _run(items, rng, pairs):
    """items: score tiles of each. pairs: a barrier for each pair of collector and sender, else one for each sender."""
    full = {(a, b): 0 for a in range(GROUPS) for b in range(GROUPS)}     # completed phases
    free, slot = [0] * GROUPS, [None] * GROUPS

    def group(g):
        """Steps of a group: yields (condition, effect); an effect that returns False has seen a wrong sum."""
        tile, sent = 0, 0
        waited = [0] * GROUPS        # sends of each group that this one goes by
        for n, m in enumerate(items):
            owner = tile % GROUPS
            mine, first = (g - owner) % GROUPS, tile
            for t in range(mine, m, GROUPS):
                yield (lambda at=first + t: at < issued[0]), (lambda at=first + t: done.add(at))
            tile += m
            if not pairs:
                before = list(waited)
                for o in range(1, min(m, GROUPS)):
                    waited[(owner + o) % GROUPS] += 1
            if mine >= m:
                continue
            if mine > 0:
                at = (owner, g) if pairs else (0, g)
                yield (lambda s=sent: s == 0 or free[g] % 2 != (s - 1) % 2), (lambda n=n: slot.__setitem__(g, n))
                yield (lambda: True), (lambda at=at: full.__setitem__(at, full[at] + 1))
                sent += 1
                continue
            for o in range(1, min(m, GROUPS)):
                b = (g + o) % GROUPS
                at, k = ((g, b), waited[b]) if pairs else ((0, b), before[b])
                if pairs:
                    waited[b] += 1
                yield (lambda at=at, k=k: full[at] % 2 != k % 2), (lambda b=b, n=n: None if slot[b] == n else False)
                yield (lambda: True), (lambda b=b: free.__setitem__(b, free[b] + 1))

    issued, done, total = [0], set(), sum(items)
    running = {g: group(g) for g in range(GROUPS)}
    at = {}
    for g in list(running):
        at[g] = next(running[g], None)
    while any(at.values()):
        while issued[0] < total and (issued[0] < GROUPS or issued[0] - GROUPS in done):
            issued[0] += 1
        ready = [g for g, s in at.items() if s and s[0]()]
        if not ready:
            return False
        # a group at a time, often the same one again: some run far ahead
        g = rng.choice(ready)
        for _ in range(rng.choice((1, 1, 2, 8))):
            if not at[g] or not at[g][0]():
                break
            if at[g][1]() is False:
                return False
            at[g] = next(running[g], None)
    return True


def _items(rng):
    return [rng.choice((1, 1, 2, 2, 3, 4, 5, 8)) for _ in range(40)]


def test_a_barrier_for_each_pair_hands_over_every_sum():
    rng = random.Random(1)
    assert all(_run(_items(rng), rng, True) for _ in range(500))


def test_a_barrier_for_each_sender_would_mix_items():
    """A collector may be an item ahead of a sender: its parity then passes by the phase before the sender's last."""
    rng = random.Random(2)
    assert not all(_run(_items(rng), rng, False) for _ in range(500))


def test_the_kernel_has_a_barrier_for_each_pair():
    with open(os.path.join(build.CSRC, "paged_weights.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "part_full[kGroups][kGroups]" in code
    assert re.search(r"mbar_arrive\(&bar\.part_full\[owner\]\[g\]\)", code)
    assert re.search(r"wait_warp\(&bar\.part_full\[g\]\[from\], \(flips >> from\) & 1,", code)
