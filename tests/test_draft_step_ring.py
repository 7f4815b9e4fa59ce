"""The hand-off of the draft step's persistent kernel (csrc/draft_step.cu), modelled on the host: one
producer stages items in order through a ring of stages, copies land in any order, groups of
consumers run at any speed, and every wait looks at a barrier's parity as the kernel's do. Each
group must get its own items, and all must end. Stages and groups are those of the kernel's four
variants, and more."""
import random

import pytest


def _run(stages, groups, fulls, items, rng):
    full, empty = [0] * fulls, [0] * stages      # completed phases
    held, landed, flying = [None] * stages, set(), []
    staged, done = 0, 0
    place, busy = list(range(groups)), [None] * groups
    while True:
        steps = []
        if staged < items and (staged < stages or empty[staged % stages] % 2 != (staged // stages - 1) % 2):
            steps.append(("stage", 0))
        steps += [("land", i) for i in range(len(flying))]
        for g in range(groups):
            if busy[g] is not None:
                steps.append(("done", g))
            elif place[g] < items and full[place[g] % fulls] % 2 != place[g] // fulls % 2:
                steps.append(("take", g))
        if not steps:
            return done == items
        what, i = rng.choice(steps)
        if what == "stage":
            held[staged % stages] = staged
            flying.append(staged)
            staged += 1
        elif what == "land":
            k = flying.pop(i)
            landed.add(k)
            full[k % fulls] += 1
        elif what == "take":
            if held[place[i] % stages] != place[i] or place[i] not in landed:
                return False
            busy[i] = place[i]
        else:
            empty[busy[i] % stages] += 1
            busy[i], done = None, done + 1
            place[i] += groups


@pytest.mark.parametrize("stages,groups", [(5, 3), (4, 3), (8, 4), (9, 4), (6, 3), (6, 4), (6, 5), (7, 2)])
def test_every_group_gets_its_items(stages, groups):
    fulls = -(-stages // groups) * groups
    rng = random.Random(stages * 10 + groups)
    assert all(_run(stages, groups, fulls, 40, rng) for _ in range(400))


def test_a_barrier_per_stage_would_mix_the_groups():
    rng = random.Random(3)
    assert not all(_run(6, 4, 6, 40, rng) for _ in range(400))
