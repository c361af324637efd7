"""CPU model of the 8-bit products' ring at its end: a CTA whose ring is not handed
back whole ends with arrivals on its barriers still to come, in memory that is the
next CTA's by then.

The loading warp waits for a stage by the parity of its barrier, which cannot tell
a phase from the one two before; the model hands stages back as late as it can, in
any order that the MMAs allow (their own), and looks at what the waits let through.
"""
import os
import re

import pytest

from tests.test_cluster_barriers import CSRC, functions


def passes(done, parity):
    """A wait for the phase of that parity, of a barrier of which `done` phases are complete."""
    return done % 2 != parity


def load(stages, items, released):
    """The loading warp's run with its tail: released(k, have) tells whether item k has been handed back when the warp waits and
    `have` items are loaded.  Returns how many releases each wait of the tail was behind, or None where a wait would not end."""
    state, parity, done = 0, 1, [0] * stages
    back = 0  # items handed back, in order

    def wait(loaded):
        nonlocal back
        while not passes(done[state], parity):
            if back == loaded:
                return False
            done[back % stages] += 1
            back += 1
        while back < loaded and released(back, loaded):
            done[back % stages] += 1
            back += 1
        return True

    for k in range(items):
        if not wait(k):
            return None
        state += 1
        if state == stages:
            state, parity = 0, parity ^ 1
    for _ in range(stages):
        if not wait(items):
            return None
        state += 1
        if state == stages:
            state, parity = 0, parity ^ 1
    return items - back


@pytest.mark.parametrize("stages", range(1, 17))
def test_the_tail_sees_every_stage_handed_back(stages):
    for items in range(0, 4 * stages + 2):
        for early in (lambda k, n: False, lambda k, n: True, lambda k, n: k % 3 != 0, lambda k, n: n - k > stages // 2):
            assert load(stages, items, early) == 0, (stages, items)


def test_every_kernel_with_such_a_ring_has_the_tail():
    found = functions(os.path.join(CSRC, "linear_f8.cu"))
    rings = {n: b for n, b, kernel in found if kernel and re.search(r"commit\(&empty\[", b)}
    assert set(rings) == {"linear_f8_kernel", "linear_f8_few_kernel", "linear_f8_pair_kernel"}
    for name, body in rings.items():
        loads, tail, close = body.find("load_2d") if "pair" not in name else body.find("f8_pair_load"), body.find("f8_ring_tail"), body.find("dealloc")
        assert 0 < loads < tail < close, name
