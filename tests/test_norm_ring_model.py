"""Model of the layer norm's copies ahead (CPU only): one thread of a block of csrc/norm.cu, its ring of
stages in shared memory, and copies that land at any time up to the wait that covers them.

A block walks its range of rows item by item. It requests groups of rows ahead, zeros past the
item's last row, and starts at the first stage again with the next item. Copies of one thread are
not ordered among each other, so none may be under way to a stage that another is requested for:
without a wait at the end of an item the zeros behind its last row could land on the next
item's first rows.
"""
import random

import pytest


def run(lo, hi, per, step, depth, seed, wait_at_end=True):
    """True if every group taken from the ring is the one that was requested for it."""
    rng = random.Random(seed)
    ring, way, count = [None] * depth, [], [0]              # way: (group's number, stage, value)

    def land(some):
        rng.shuffle(way)
        for c in list(way):
            if some(c):
                way.remove(c)
                ring[c[1]] = c[2]

    def wait(n):                                            # all but the last n groups
        land(lambda c: c[0] < count[0] - n)

    r0 = lo
    while r0 < hi:
        end = min(hi, (r0 // per + 1) * per)
        put = got = 0

        def request(base):
            nonlocal put
            way.append((count[0], put, base if base < end else "zeros"))
            count[0] += 1
            put = (put + 1) % depth
            land(lambda c: rng.random() < 0.3)

        for i in range(depth - 1):
            request(r0 + i * step)
        for base in range(r0, end, step):
            request(base + (depth - 1) * step)
            wait(depth - 1)
            if ring[got] != base:
                return False
            got = (got + 1) % depth
        if wait_at_end:
            wait(0)
        r0 = end
    return True


CASES = [(0, 40, 10, 2), (7, 61, 20, 4), (0, 12, 1, 2), (3, 30, 9, 16), (0, 50, 50, 8)]


@pytest.mark.parametrize("depth", [1, 2, 3, 4])
def test_every_group_is_its_own(depth):
    assert all(run(*case, depth, seed) for case in CASES for seed in range(200))


@pytest.mark.parametrize("depth", [2, 3, 4])
def test_copies_left_under_way_at_the_end_of_an_item_are_caught(depth):
    for case in CASES[:2]:
        assert not all(run(*case, depth, seed, wait_at_end=False) for seed in range(200)), case
    # one group an item, or one item a range, never meets it
    assert all(run(*case, depth, seed, wait_at_end=False) for case in CASES[2:] for seed in range(200))
