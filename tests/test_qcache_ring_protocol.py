"""A model of the ring that each warp of the attention over a 4-bit cache fills for itself (few rows): two slots with a barrier
each, copies that run two slices ahead within a piece and start a piece's first ones before the piece before is put
together.

The model replays the loads and waits of a warp with copies that land late, and one that does not land before a bounded wait
gives up.  A barrier's phase completes on one arrival and the bytes that it announces; an arrival in a phase that has
had its own already, or a copy into a slot that another is still under way to, is an error.  A warp that went on loading
after it gave up must fail.
"""
import random

import pytest

STAGES = 2


class Slot:
    def __init__(self):
        self.armed = self.landed = 0

    def arm(self):
        assert self.armed == self.landed, "an arrival in a phase that has had its own"
        self.armed += 1


def replay(pieces, seed, lost=None, stop=True):
    """The slices per piece of one warp; `lost`: the copy (counted as they start) that lands only after the limit.  The slices
    that the warp computed from copies that had landed."""
    rng = random.Random(seed)
    slots, flights, ok, used, started, sound = [Slot() for _ in range(STAGES)], [], True, 0, 0, []

    def load(count):
        nonlocal started
        if stop and not ok:
            return
        slots[count % STAGES].arm()
        flights.append((count % STAGES, started == lost))
        started += 1

    def land(slot):
        """The copies into this slot land, others perhaps; True if they did."""
        for f in list(flights):
            if not f[1] and (f[0] == slot or rng.random() < 0.5):
                flights.remove(f)
                slots[f[0]].landed += 1
        return all(f[0] != slot for f in flights)

    def first(n):
        for i in range(min(n, STAGES)):
            load(used + i)

    first(pieces[0])
    for p, n in enumerate(pieces):
        for j in range(n):
            slot = used % STAGES
            if ok:
                ok = land(slot) and slots[slot].landed == used // STAGES + 1
            if ok:
                sound.append((p, j))
            if j + STAGES < n:
                load(used + STAGES)
            used += 1
        if p + 1 < len(pieces):
            first(pieces[p + 1])
    return ok, sound


PIECES = [[1], [2], [3], [9], [4, 4], [1, 1, 1], [0, 3, 0, 1], [5, 0, 2, 7], [2, 3, 2, 5]]


@pytest.mark.parametrize("pieces", PIECES)
def test_every_slice_is_computed_from_its_own_copy(pieces):
    for seed in range(50):
        ok, sound = replay(pieces, seed)
        assert ok and sound == [(p, j) for p, n in enumerate(pieces) for j in range(n)]


@pytest.mark.parametrize("pieces", PIECES)
def test_a_copy_that_does_not_come_ends_the_loads(pieces):
    for lost in range(sum(pieces)):
        for seed in range(50):
            ok, sound = replay(pieces, seed, lost)
            assert not ok and len(sound) == lost


def test_loading_on_after_giving_up_meets_an_open_phase():
    failed = 0
    for seed in range(20):
        try:
            replay([9], seed, 0, stop=False)
        except AssertionError:
            failed += 1
    assert failed == 20
