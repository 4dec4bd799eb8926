"""CPU model of the pair GEMM's stage release (gemm.cuh): the coordinator warp arrives at named barrier it % TB for
every k-stage, the MMA warp waits there (64 threads: 32 of each) and commits the stage's MMAs.  After a failure the
coordinator releases the rest of its tile without waiting for data.  However the two warps interleave, the MMA
warp never waits at a barrier for good.  A change to the hand-off must be mirrored here."""
import random

import pytest

TB = 3


class NamedBarrier:
    """64 threads complete a generation; a warp that arrives twice in one generation completes it alone."""

    def __init__(self):
        self.count, self.generation = 0, 0

    def arrive(self):
        self.count += 32
        if self.count == 64:
            self.count, self.generation = 0, self.generation + 1


def run(rng, tiles, stages, fail_at, mma_leaves_after, paced):
    """False where the MMA warp is left waiting.  `fail_at`: the stage (over all tiles) whose data never come;
    `mma_leaves_after`: a tile after which the MMA warp sees an abort of another warp, or None."""
    bars, committed = [NamedBarrier() for _ in range(TB)], [0]
    state = {"ok": True, "left": False}

    def coordinator():
        it = 0
        for _ in range(tiles):
            if not state["ok"]:
                return
            for _ in range(stages):
                if it >= fail_at:
                    state["ok"] = False
                # the scale buffer (before a failure), or (paced) the wait after it
                if it >= TB and (state["ok"] or paced):
                    while committed[0] <= it - TB:
                        if state["left"]:
                            return
                        yield
                bars[it % TB].arrive()
                yield
                it += 1

    def mma():
        it = 0
        for tile in range(tiles):
            for _ in range(stages):
                bar = bars[it % TB]
                generation = bar.generation
                bar.arrive()
                while bar.generation == generation:
                    yield
                it += 1
                committed[0] = it
                yield
            if not state["ok"] or tile == mma_leaves_after:
                state["left"] = True
                return

    warps = {"coordinator": coordinator(), "mma": mma()}
    idle = 0
    while warps and idle < 400:
        name = rng.choice(sorted(warps))
        before = (committed[0], [(b.count, b.generation) for b in bars])
        try:
            next(warps[name])
        except StopIteration:
            del warps[name]
        idle = 0 if before != (committed[0], [(b.count, b.generation) for b in bars]) else idle + 1
    return "mma" not in warps


@pytest.mark.parametrize("stages", [1, 2, 3, 4, 7, 20])
def test_the_mma_warp_always_leaves(stages):
    for seed in range(60):
        rng = random.Random(seed)
        tiles = rng.randint(1, 4)
        fail_at = rng.randint(0, tiles * stages)
        leaves = rng.choice([None, rng.randrange(tiles)])
        if leaves is not None and fail_at > (leaves + 1) * stages:
            fail_at = (leaves + 1) * stages  # (the abort ends the coordinator's waits too)
        assert run(rng, tiles, stages, fail_at, leaves, paced=True), (seed, stages)


def test_the_model_sees_the_lapped_ring():
    assert not all(run(random.Random(seed), 2, 20, 1, None, paced=False) for seed in range(60))
