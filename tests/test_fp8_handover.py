"""Who may touch what when in the block-scaled 8-bit product, on the CPU: a model of one CTA's warps with vector clocks.

Two warps write the products of the scales to a ring; an issuer multiplies; the epilogue's warps read both, and give the
ring's places back a group at a time.  Clocks travel over barriers that are arrived on with release, not over relaxed
arrivals, nor over the MMAs' commits.  Every access to the ring and to the tiles' coordinates must be ordered behind the
ones before it, whatever the order the warps run in.
"""
import random

import pytest

EPILOGUES = 4
RING, GROUP, TILES = 8, 4, 16


class _Race(Exception):
    pass


class _Barrier:
    def __init__(self, count, actors):
        self.count, self.left, self.phases = count, count, 0
        self.clock, self.ended = [0] * actors, []

    def arrive(self, clock=None):
        if clock is not None:  # a release
            self.clock = [max(a, b) for a, b in zip(self.clock, clock)]
        self.left -= 1
        if self.left == 0:
            self.ended.append(self.clock)
            self.left, self.phases = self.count, self.phases + 1


class _Place:
    """Memory that one side writes and the other reads."""

    def __init__(self):
        self.writes, self.reads, self.holds = {}, {}, {}

    def write(self, actor, clock, value):
        if any(clock[a] < at for a, at in self.reads.items()):
            raise _Race("overwritten before it was read")
        self.writes[actor], self.holds[actor] = clock[actor], value

    def read(self, actor, clock, value):
        if any(clock[a] < at for a, at in self.writes.items()):
            raise _Race("read before it was written")
        if any(v != value for v in self.holds.values()):
            raise _Race("another stage's")
        self.reads[actor] = clock[actor]


def _run(slots, blocks, stages, ordered, rng, places=TILES):
    """slots accumulators, tiles of `blocks` stages; ordered: the epilogue's arrivals on `read` release."""
    actors = 3 + EPILOGUES  # two warps with scales, the issuer, the epilogue
    clocks = [[0] * actors for _ in range(actors)]
    full = [_Barrier(3, actors) for _ in range(slots)]
    empty, read = ([_Barrier(EPILOGUES, actors) for _ in range(n)] for n in (slots, 2))
    factors, tiles = [_Place() for _ in range(RING)], [_Place() for _ in range(places)]

    def wait(me, bar, phase):
        while bar.phases <= phase:
            yield
        assert bar.phases == phase + 1, "a phase later: the parity no longer tells"
        clocks[me] = [max(a, b) for a, b in zip(clocks[me], bar.ended[phase])]

    def step(me):
        clocks[me][me] += 1
        return clocks[me]

    def scales(me):
        for n in range(stages):
            if n >= RING and n % GROUP == 0:
                yield from wait(me, read[n // GROUP % 2], n // RING - 1)
            if n >= slots:
                yield from wait(me, full[n % slots], n // slots - 1)
            factors[n % RING].write(me, step(me), n)
            if me == 0 and n % blocks == 0:
                tiles[n // blocks % places].write(me, step(me), n // blocks)
            yield
            full[n % slots].arrive(step(me))

    def issuer(me):
        for n in range(stages):
            if n >= slots:
                yield from wait(me, empty[n % slots], n // slots - 1)
            yield
            full[n % slots].arrive()

    def epilogue(me):
        for n in range(stages):
            if n % GROUP == 0 and n > 0:
                read[(n // GROUP - 1) % 2].arrive(step(me) if ordered else None)
                yield
            yield from wait(me, full[n % slots], n // slots)
            factors[n % RING].read(me, step(me), n)
            yield
            empty[n % slots].arrive()
            yield
            if n % blocks == blocks - 1:
                tiles[n // blocks % places].read(me, step(me), n // blocks)

    running = [scales(0), scales(1), issuer(2)] + [epilogue(3 + i) for i in range(EPILOGUES)]
    weight = [rng.choice([1, 1, 5, 25]) for _ in running]
    for _ in range(2000 * stages):
        i = rng.choices(range(len(running)), weight)[0]
        try:
            next(running[i])
        except StopIteration:
            del running[i], weight[i]
            if not running:
                return
    raise AssertionError("a wait that does not end")


@pytest.mark.parametrize("slots", [2, 4])
@pytest.mark.parametrize("blocks", [1, 2, 3, 7])
def test_every_access_is_ordered(slots, blocks):
    for seed in range(10):
        _run(slots, blocks, 84, True, random.Random(seed))


@pytest.mark.parametrize("slots", [2, 4])
def test_the_model_sees_places_that_nobody_gives_back(slots):
    with pytest.raises(_Race):
        _run(slots, 1, 84, False, random.Random(0))


def test_the_model_sees_too_few_places_for_tiles():
    with pytest.raises(_Race):
        for seed in range(40):
            _run(4, 1, 84, True, random.Random(seed), places=3)
