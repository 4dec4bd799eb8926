"""CPU model of the gated residual epilogue's tile ring (gemm.cuh, one epilogue warp): three shared-memory tiles
take the four residual chunks of an output tile by asynchronous copies, each tile under one barrier.  Whenever the
kernel gives up (its abort flag is set by another warp, or this warp's accumulator does not come) no barrier is
armed while its phase is open, no tile is read or written while a copy into it is in flight, and none is in flight
when the CTA exits.  A change to the ring must be mirrored here."""
import itertools

import pytest


class Hazard(Exception):
    pass


class Ring:
    """Three barriers (one arrival a phase) and the copies in flight, which land as soon as a wait lets them."""

    def __init__(self):
        self.phase, self.armed = [0, 0, 0], [False] * 3

    def load(self, slot):
        if self.armed[slot]:
            raise Hazard("armed twice")
        self.armed[slot] = True

    def wait(self, slot, parity, stays):
        """Until the phase of this parity is complete (the current one has the other); a wait that the abort flag
        ends (`stays` false) returns before the copy has landed."""
        while self.phase[slot] & 1 == parity:
            assert self.armed[slot], "a wait for a phase that nothing completes"
            if not stays:
                return
            self.armed[slot], self.phase[slot] = False, self.phase[slot] + 1

    def touch(self, slot):
        if self.armed[slot]:
            raise Hazard("tile used while a copy is in flight")


def warp(tiles, abort_at, accumulator_lost, heeds_abort):
    """One warp over `tiles` output tiles.  From wait number `abort_at` on the abort flag is set; the accumulator of
    tile `accumulator_lost` never comes."""
    ring, res_tiles, n, aborted = Ring(), 0, 0, False
    for tile in range(tiles):
        for k in range(3):
            ring.load(k % 3)
        if tile == accumulator_lost:
            for k in range(3):
                ring.wait(k, 0 if k == 0 else res_tiles & 1, True)
            break
        for k in range(4):
            aborted |= n == abort_at
            parity = (1 if k == 3 else 0) if k % 3 == 0 else res_tiles & 1
            ring.wait(k % 3, parity, not (aborted and heeds_abort))
            n += 1
            ring.touch(k % 3)
            if k == 1:
                ring.load(0)
            if k == 3:
                res_tiles += 1
    if any(ring.armed):
        raise Hazard("a copy in flight at the exit")


@pytest.mark.parametrize("tiles", [1, 2, 3, 6])
def test_no_copy_is_left(tiles):
    for abort_at, lost in itertools.product((None, *range(4 * tiles)), (None, *range(tiles))):
        warp(tiles, abort_at, lost, heeds_abort=False)


def test_the_model_sees_the_hazard():
    """Waits that the abort flag ends leave copies in flight."""
    for tiles in (1, 2, 3):
        for abort_at in range(4 * tiles):
            with pytest.raises(Hazard):
                warp(tiles, abort_at, None, heeds_abort=True)
