"""How the waves of an attention workgroup hand over their parts of rows
(csrc_decode/tq_attn_slots.h), checked on the CPU.

A wave first marks its slots empty, later fills the ones in which it leaves a part,
and only then meets the others at a barrier: between the waves nothing is ordered
before it.  This test compiles the header's arithmetic with g++ and replays every
order of the waves' stores for both forms of the kernel: at the barrier each
published part has to be there, and no other.
"""

import itertools
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_mixed_precision_amd", "csrc_decode")

DRIVER = r"""
#include <cstdio>
#include "tq_attn_slots.h"
int main() {
  std::printf("%d %d %d\n", tq::kAttnWaves, tq::kAttnParts, tq::kAttnSlots);
  for (int w = 0; w < tq::kAttnWaves; ++w)
    for (int p = 0; p < tq::kAttnParts; ++p) {
      const int s = tq::attn_slot(w, p);
      std::printf("%d %d %d %d %d\n", w, p, s, tq::attn_sums_at(false, s), tq::attn_sums_at(true, s));
    }
}
"""


@pytest.fixture(scope="module")
def slots(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("slots")
    (d / "drv.cpp").write_text(DRIVER)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}", str(d / "drv.cpp"), "-o",
                    str(d / "drv")], check=True)
    out = subprocess.run([str(d / "drv")], capture_output=True, text=True, check=True).stdout
    rows = [[int(x) for x in line.split()] for line in out.strip().splitlines()]
    waves, parts, count = rows[0]
    assert len(rows) == 1 + waves * parts and count == waves * parts
    return dict(waves=waves, parts=parts, count=count,
                slot={(r[0], r[1]): r[2] for r in rows[1:]},
                sums={False: {r[2]: r[3] for r in rows[1:]}, True: {r[2]: r[4] for r in rows[1:]}})


def lost(marks, fills):
    """The first (mark, fill) pair whose order is open and matters, else None: a mark
    of one wave and a part of another in the same slot, or two parts there.  Waves are
    not ordered against each other, so any such pair can come in either order; without
    one, every order of all stores ends the same."""
    for a, b in itertools.permutations(range(len(marks)), 2):
        if set(marks[a]) & set(fills[b]):
            return "mark", a, b
        if set(fills[a]) & set(fills[b]):
            return "part", a, b
    return None


def replay(order, marks, fills):
    """Contents of the slots after the waves' programs (marks, then fills) were run
    in this order of wave numbers."""
    state, at = {}, [0] * len(marks)
    for w in order:
        if at[w] < len(marks[w]):
            state[marks[w][at[w]]] = -1
        else:
            state[fills[w][at[w] - len(marks[w])]] = w
        at[w] += 1
    return state


@pytest.mark.parametrize("direct", [False, True])
def test_every_order_of_the_waves_keeps_every_part(slots, direct):
    W, parts = slots["waves"], slots["parts"]
    marks = [[slots["slot"][w, p] for p in range(parts)] for w in range(W)]
    used = 1 if direct else parts  # a workgroup with one row leaves no second parts
    fills = [[slots["slot"][w, p] for p in range(used)] for w in range(W)]
    assert sorted(s for m in marks for s in m) == list(range(slots["count"]))  # all are marked
    assert lost(marks, fills) is None
    # every order of two waves' programs, each pair in turn
    for a, b in itertools.combinations(range(W), 2):
        m, f = [marks[a], marks[b]], [fills[a], fills[b]]
        steps = [len(m[0]) + len(f[0]), len(m[1]) + len(f[1])]
        for first in itertools.combinations(range(sum(steps)), steps[0]):
            order = [0 if i in first else 1 for i in range(sum(steps))]
            state = replay(order, m, f)
            assert all(state[s] == w for w in range(2) for s in f[w])
            assert sum(v == -1 for v in state.values()) == 2 * (parts - used)
    # the sums of two parts never share a place, and the places are packed
    places = [slots["sums"][direct][s] for f in fills for s in f]
    assert sorted(places) == list(range(W * used))


def test_the_replay_finds_a_foreign_mark():
    """A mapping in which one wave marks the slot that another fills is caught."""
    marks, fills = [[2 * w, 2 * w + 1] for w in range(4)], [[w] for w in range(4)]
    assert lost(marks, fills) == ("mark", 0, 1)
    assert replay([0, 0, 1, 1, 1, 0], marks[:2], fills[:2])[1] == 1
    assert replay([1, 1, 1, 0, 0, 0], marks[:2], fills[:2])[1] == -1  # wave 1's part is gone
