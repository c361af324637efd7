"""CPU model of the tree attention kernel's ring: who may wait for what.

One ring of slots carries K and V of a CTA's segments in the order of ta_item
(K0, K1, V0, K2, V1, ...), NS slots an operand.  With box copies one warp fills
K's items and another V's; the MMA warp takes the items in order.  A loader
waits for a free slot by parity, which cannot tell the round it means from the
one two before.  The model walks every interleaving of the three roles and
reports a wait that parity lets through too early, and a state in which nobody
can go on.  Shapes and order come from csrc/tree_shape.h, compiled here.
"""
import itertools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_weight_reconstruction_wl_gb300", "csrc")

SRC = r"""
#include <cstdio>
#include "tree_shape.h"
using namespace wl;
template <bool e, int d, int r> void shape()
{
    using Z = TaShape<e, d, r>;
    std::printf("shape %d %d %d %d %d %d\n", (int)e, d, r, Z::SLOTS, Z::NS, (int)Z::PACED);
}
int main()
{
    shape<true, 128, 16>(); shape<true, 128, 32>(); shape<true, 128, 64>();
    shape<true, 256, 16>(); shape<true, 256, 32>(); shape<true, 256, 64>();
    shape<false, 128, 16>(); shape<false, 128, 32>(); shape<false, 128, 64>();
    shape<false, 256, 16>(); shape<false, 256, 32>(); shape<false, 256, 64>();
    for (int n = 1; n <= 6; ++n)
        for (int r = 0; r < n; ++r) std::printf("item %d %d %d %d\n", n, r, ta_item(r, n, false), ta_item(r, n, true));
}
"""


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "s.cpp").write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "s.cpp"), "-o", str(d / "s")], check=True)
    shapes, order = {}, {}
    for line in subprocess.run([str(d / "s")], capture_output=True, text=True, check=True).stdout.splitlines():
        w = line.split()
        v = [int(x) for x in w[1:]]
        if w[0] == "shape":
            shapes[("e4m3" if v[0] else "bf16", v[1], v[2])] = dict(slots=v[3], ns=v[4], paced=bool(v[5]))
        else:
            order[(v[0], v[1])] = (v[2], v[3])
    return shapes, order


def passes(done, use):
    """A parity wait for completion `use` (from 0) of a barrier of which `done` phases are complete."""
    return done % 2 == (use + 1) % 2


class Ring:
    """The items of a sequence of segments: per loader, and in the order of the MMA warp."""

    def __init__(self, order, lengths, ns):
        self.mine = ([], [])      # items of K's and of V's warp, in the order it fills them
        self.head = ({}, {})      # ... the first item of a segment -> items of the other warp that come first, if in step
        at = 0
        for n in lengths:
            for r in range(n):
                for v in (0, 1):
                    self.mine[v].extend(at + order[(n, r)][v] * ns + s for s in range(ns))
            if at:
                self.head[0][at] = at - 1                                    # V's last of the segment before
            self.head[1][at + order[(n, 0)][1] * ns] = at + order[(n, min(n, 2) - 1)][0] * ns + ns - 1
            at += 2 * n * ns
        self.items = at
        # [item of V, items consumed once the scores of its tile are there, last tile of its segment]
        self.values = []
        at = 0
        for n in lengths:
            self.values += [(at + order[(n, r)][1] * ns + s, at + (order[(n, r)][0] + 1) * ns, r == n - 1) for r in range(n) for s in range(ns)]
            at += 2 * n * ns
        assert sorted(self.mine[0] + self.mine[1]) == list(range(at))

    def faults(self, slots, paced, look="none", states=None):
        """Walks every reachable (K's place, V's place, items consumed).

        look: the tiles whose V a softmax warp waits for on its own, by the full barrier's parity, between its
        scores and its weights (the MMA warp cannot take that V before): "none", a segment's "last", "all"."""
        bad, seen, todo = set(), {(0, 0, 0)}, [(0, 0, 0)]
        while todo:
            state = todo.pop()
            k, v, c = state
            nxt = []
            for y, scored, last in self.values:
                if look == "none" or (look == "last" and not last) or not scored <= c <= y:
                    continue
                # rounds of the slot that have landed: all consumed ones, or also the one in flight
                issued = sum(i % slots == y % slots for i in self.mine[0][:k] + self.mine[1][:v])
                for landed in {len(range(y % slots, c, slots)), issued}:
                    if passes(landed, y // slots) and landed != y // slots + 1:
                        bad.add(("takes another round for V", y))
            for w, place in ((0, k), (1, v)):
                if place == len(self.mine[w]):
                    continue
                x = self.mine[w][place]
                other = self.mine[1 - w][:(v, k)[w]]
                if paced and self.head[w].get(x, -1) >= 0 and self.head[w][x] not in other:
                    continue
                # items of this slot consumed: x % slots, + slots, ... below c
                done = len(range(x % slots, c, slots))
                if passes(done, x // slots - 1):
                    if x >= slots and c <= x - slots:
                        bad.add(("fills a slot in use", x))
                        continue
                    nxt.append((k + 1, v, c) if w == 0 else (k, v + 1, c))
            if c in self.mine[0][:k] or c in self.mine[1][:v]:
                nxt.append((k, v, c + 1))
            if states is not None:
                states.add(state)
            if not nxt and c < self.items:
                bad.add(("stuck", state))
            for s in nxt:
                if s not in seen:
                    seen.add(s)
                    todo.append(s)
        return bad


LENGTHS = [s for k in (1, 2, 3) for s in itertools.product((1, 2, 3, 4, 5), repeat=k)] + [(1, 1, 1, 3, 1, 2, 1), (6, 1, 6, 2), (2, 2, 2, 2, 2)]


def test_no_loader_fills_a_slot_in_use(compiled):
    """Every shape, over segments of all small lengths."""
    shapes, order = compiled
    for ring in {(z["slots"], z["ns"], z["paced"]) for z in shapes.values()}:
        for lengths in LENGTHS:
            bad = Ring(order, lengths, ring[1]).faults(ring[0], ring[2])
            assert not bad, (ring, lengths, sorted(bad)[:4])


def test_shapes_that_need_it_keep_their_warps_in_step(compiled):
    """Without the step some shape overwrites a slot (the model is not vacuous); only those shapes pay for it."""
    shapes, order = compiled
    for name, z in shapes.items():
        free = any(Ring(order, lengths, z["ns"]).faults(z["slots"], False) for lengths in LENGTHS)
        assert free == z["paced"], (name, z)
    assert shapes[("bf16", 256, 64)]["paced"]


@pytest.mark.parametrize("lengths", [(1, 3), (2, 3), (3, 3), (6, 4)])
def test_four_slots_of_two_an_operand(compiled, lengths):
    ring = Ring(compiled[1], lengths, 2)
    assert any(f[0] == "fills a slot in use" for f in ring.faults(4, False))
    assert not ring.faults(4, True)


def test_waits_of_the_softmax_warps_for_v(compiled):
    """They look at a last tile's V in every shape; at any tile's only where the ring holds three operands' slots."""
    shapes, order = compiled
    some = LENGTHS[:155:3] + LENGTHS[-3:]
    for ring in {(z["slots"], z["ns"], z["paced"]) for z in shapes.values()}:
        for lengths in some:
            assert not Ring(order, lengths, ring[1]).faults(*(ring[0], ring[2]), look="last"), (ring, lengths)
        wrong = any(Ring(order, lengths, ring[1]).faults(*(ring[0], ring[2]), look="all") for lengths in some)
        assert wrong == (ring[0] < 3 * ring[1]), ring


def test_what_is_in_flight_can_be_waited_for_at_any_point(compiled):
    """Where every role stops, the last item copied to a slot is the one whose landing its full barrier's parity
    tells, and only that one can be in flight."""
    shapes, order = compiled
    for slots, ns, paced in {(z["slots"], z["ns"], z["paced"]) for z in shapes.values()}:
        for lengths in LENGTHS[:155:2] + LENGTHS[-3:]:
            ring = Ring(order, lengths, ns)
            states = set()
            assert not ring.faults(slots, paced, states=states)
            for k, v, c in states:
                copied = ring.mine[0][:k] + ring.mine[1][:v]
                for s in range(slots):
                    mine = sorted(i for i in copied if i % slots == s)
                    assert mine == list(range(s, s + slots * len(mine), slots))  # no round left out
                    assert all(i < c for i in mine[:-1])                         # all but the last consumed
