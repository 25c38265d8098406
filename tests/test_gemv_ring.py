"""The stage ring of the few-row NVFP4 product, as a model of its barriers on the CPU.

The roles are those of nvfp4_gemv_kernel: a loader, an MMA warp, and two sets of four warps that
move scales, each its own stages, and look at the phases of the others'.  A barrier wait sees the
parity of a phase and nothing else, so a role that is a turn of the ring behind is let through, or held,
by the wrong fill.  How many arrivals a refill waits for, and whether the set that only looks is
among them, is read from the kernel's source; the schedules are random, with one warp slower than the rest."""
import os
import random
import re

import pytest

import video_dit_dynamic_token_b200 as pkg

SRC = os.path.join(os.path.dirname(pkg.__file__), "csrc", "nvfp4_gemv.cuh")


class _Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0            # completed phases

    def arrive(self):
        assert self.left > 0
        self.left -= 1
        if self.left == 0:
            self.phase += 1
            self.left = self.count

    def passed(self, parity):
        return (self.phase - 1) & 1 == parity


def _simulate(n, stages, arrivals, look_arrives, slow, rng):
    """Runs the roles over n stages; returns a description of the first fault, or None."""
    full = [_Barrier(1) for _ in range(stages)]
    empty = [_Barrier(arrivals) for _ in range(stages)]
    sf = [_Barrier(4) for _ in range(stages)]
    holds = [None] * stages       # the stage whose data a slot has
    flying = []                   # asynchronous completions: loads and commits
    faults = []

    def fill(i):
        holds[i % stages] = i
        full[i % stages].arrive()

    def loader():
        for i in range(n):
            if i >= stages:
                yield lambda i=i: empty[i % stages].passed((i // stages - 1) & 1)
            flying.append(lambda i=i: fill(i))

    def mma():
        for i in range(n):
            s, ph = i % stages, (i // stages) & 1
            yield lambda: full[s].passed(ph)
            yield lambda: sf[s].passed(ph)
            if holds[s] != i:
                faults.append(f"MMA of stage {i} reads stage {holds[s]}")
            flying.append(lambda s=s: empty[s].arrive())

    def scales(which):
        for i in range(n):
            s, ph = i % stages, (i // stages) & 1
            yield lambda: full[s].passed(ph)
            if i & 1 != which:
                if look_arrives:
                    empty[s].arrive()
                continue
            if holds[s] != i:
                faults.append(f"scales of stage {i} are those of stage {holds[s]}")
            sf[s].arrive()

    roles = [loader(), mma()] + [scales(w // 4) for w in range(8)]
    waits = [next(r, "done") for r in roles]
    while any(w != "done" for w in waits):
        ready = [k for k, w in enumerate(waits) if w != "done" and w()]
        if not ready and not flying:
            return "stuck: " + ", ".join(str(k) for k, w in enumerate(waits) if w != "done")
        others = [k for k in ready if k != slow]
        if flying and (not others or rng.random() < 0.5):
            flying.pop(rng.randrange(len(flying)))()
        elif others and rng.random() < 0.98:
            k = rng.choice(others)
            waits[k] = next(roles[k], "done")
        elif ready:
            k = rng.choice(ready)
            waits[k] = next(roles[k], "done")
        if faults:
            return faults[0]
    return None


def _protocol():
    src = open(SRC).read()
    arrivals = sum(int(x) for x in re.search(r"mbar_init\(&bar_empty\[s\], ([\d +]+)\)", src).group(1).split("+"))
    look = re.search(r"if \(\(i & 1\) != set\) (.*?)continue;", src, re.S).group(1)
    return arrivals, "mbar_arrive(&bar_empty[s])" in look


@pytest.mark.parametrize("stages", [3, 4, 5])
def test_no_schedule_passes_a_turn_of_the_ring(stages):
    arrivals, look = _protocol()
    for seed in range(300):
        rng = random.Random(seed)
        slow = rng.choice([None, 0, 1] + list(range(2, 10)))
        fault = _simulate(rng.randint(1, 40), stages, arrivals, look, slow, rng)
        assert fault is None, f"seed {seed}, slow role {slow}: {fault}"


def test_the_model_sees_a_missing_arrival():
    """A refill that waits for the MMA alone: a looking warp that is late is left behind."""
    found = [_simulate(30, 3, 1, False, 2 + seed % 8, random.Random(seed)) for seed in range(300)]
    assert any(found)
