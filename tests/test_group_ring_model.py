"""The copy ring of the grouped-row K pass, as a model of its barriers (no GPU needed).

Three producer warps deal out a step's boxes among themselves and follow the ring by
the parity of its barriers; a step may have fewer boxes than there are producers.  The
model takes the number of arrivals that fill a slot from the kernel's source and lets
one producer lag for as long as the others can run: each wait has to end all the same.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_compressed_kv_star_b200", "csrc")


def _source():
    text = open(os.path.join(CSRC, "group_kernels.cuh")).read()
    producers = int(re.search(r"constexpr int kGKProd = (\d+);", text).group(1))
    start = text.index("group_kpass_kernel(")
    body = text[start:text.index("group_vpass_kernel(", start)]
    count = re.search(r"mbar_init\(&full\[s\], (\w+)\)", body).group(1)
    return producers, producers if count == "kGKProd" else int(count)


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.bytes, self.phase = count, count, 0, 0

    def arrive(self, tx=0):
        self.bytes += tx
        self.pending -= 1
        self._flip()

    def land(self, n):
        self.bytes -= n
        self._flip()

    def _flip(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count

    def passed(self, parity):   # the wait's own test: has the phase of this parity completed?
        return (self.phase & 1) != parity


def run(steps, slots, producers, arrivals, pick):
    """True if every warp comes to its end; `pick` chooses among the warps that can go on."""
    full, empty = [Barrier(arrivals) for _ in range(slots)], [Barrier(1) for _ in range(slots)]

    def producer(pid):
        for k, nb in enumerate(steps):
            s, u = k % slots, k // slots
            if u > 0:
                yield lambda: empty[s].passed((u - 1) & 1)
            mine = len(range(pid, nb, producers))
            if arrivals > 1:
                full[s].arrive(mine)
            elif pid == 0:
                full[s].arrive(nb)
            for _ in range(mine):
                yield lambda: True
                full[s].land(1)

    def consumer():
        for k in range(len(steps)):
            s, u = k % slots, k // slots
            yield lambda: full[s].passed(u & 1)
            empty[s].arrive()

    warps = dict(enumerate([producer(p) for p in range(producers)] + [consumer()]))
    waits = {w: next(g, None) for w, g in warps.items()}
    while any(x is not None for x in waits.values()):
        can = [w for w, x in waits.items() if x is not None and x()]
        if not can:
            return False
        w = pick(can)
        waits[w] = next(warps[w], None)
    return True


CASES = [[1] * 37, [2] * 29, [1] * 9 + [8] * 5, [8] * 6 + [1] * 21 + [8] * 3, [1] * 8, [3, 1, 2, 8, 1, 1, 1, 5] * 4]


@pytest.mark.parametrize("slots", [2, 3, 8])
@pytest.mark.parametrize("lagging", [0, 1, 2])
def test_a_lagging_producer_is_waited_for(slots, lagging):
    producers, arrivals = _source()
    for steps in CASES:
        assert run(steps, slots, producers, arrivals, lambda can: max(can, key=lambda w: (w != lagging, w))), (steps, slots)


def test_any_order_ends():
    producers, arrivals = _source()
    rng = random.Random(8)
    for _ in range(300):
        steps = [rng.choice((1, 1, 1, 2, 3, 8)) for _ in range(rng.randint(1, 60))]
        slow = rng.randrange(producers)
        pick = lambda can: rng.choice([w for w in can if w != slow] or can) if rng.random() < 0.97 else rng.choice(can)
        assert run(steps, rng.randint(2, 8), producers, arrivals, pick), steps


def test_the_model_sees_the_lap():
    """One arrival for all producers, as a check of the model itself."""
    ok = [run(steps, 3, 3, 1, lambda can: max(can, key=lambda w: (w != 2, w))) for steps in CASES]
    assert not all(ok)
