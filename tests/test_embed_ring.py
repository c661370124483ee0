"""The bookkeeping of the ring through which the embedding gradient's sums take
their rows, on the host: a small program walks items through it as the kernel
does, over barriers of which one never completes, and counts what was done."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "embed_ring.cuh"

// Two barriers; the batch number `late` (in the order asked for) never arrives, or only at the second wait for it.
struct Bars {
    int asked[2] = {0, 0}, ended[2] = {0, 0}, order = 0, late = -1, slot_late = -1, waits_late = 0, arrives_at = 0;
    bool asked_in_flight = false, parity_wrong = false;
    void ask(int s)
    {
        if (asked[s] != ended[s]) asked_in_flight = true; // the slot's batch has not been waited for
        if (order++ == late) slot_late = s;
        ++asked[s];
    }
    bool wait(int s, uint32_t parity)
    {
        if ((uint32_t)(ended[s] & 1) != parity) parity_wrong = true;
        if (asked[s] == ended[s]) return false; // nothing is on its way: a wait without an end
        if (s == slot_late) {
            if (++waits_late != arrives_at) return false;
        }
        ++ended[s];
        return true;
    }
};

int main(int argc, char **argv)
{
    const int kStages = 8, kBatch = 4, slots = kStages / kBatch;
    Bars bars;
    bars.late = atoi(argv[1]);
    bars.arrives_at = atoi(argv[2]);
    ap::RingState state;
    int summed = 0, spoiled = 0, flags = 0, items = argc - 3;
    auto wait = [&](int s, uint32_t parity) { return bars.wait(s, parity); };
    auto fetch = [&](int live, int r0) {
        const int slot = r0 / kBatch % slots;
        if (live - r0 <= 0 || !state.arm(slot)) return;
        bars.ask(slot);
    };
    int ahead = atoi(argv[3]);
    for (int r = 0; r < kStages; r += kBatch) fetch(ahead, r);
    for (int it = 0; it < items; ++it) {
        const int live = ahead;
        if (it + 1 < items) ahead = atoi(argv[3 + it + 1]);
        for (int r0 = 0; r0 < live; r0 += kBatch) {
            const bool was_lost = state.lost;
            if (!state.take(r0 / kBatch % slots, wait)) {
                flags += !was_lost;
                spoiled += live - r0;
                break;
            }
            summed += live - r0 < kBatch ? live - r0 : kBatch;
            fetch(live, r0 + kStages);
        }
        if (it + 1 < items)
            for (int r = 0; r < kStages; r += kBatch) fetch(ahead, r);
    }
    const int open = bars.asked[0] - bars.ended[0] + bars.asked[1] - bars.ended[1];
    printf("%d %d %d %d %d %d %d\n", summed, spoiled, flags, open, bars.waits_late, bars.asked_in_flight, bars.parity_wrong);
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "activation_paging_gb300", "csrc"), str(d / "ring.cpp"), "-o", str(d / "ring")],
                   check=True)

    def run(late, arrives_at, lives):
        out = subprocess.run([str(d / "ring"), str(late), str(arrives_at)] + [str(v) for v in lives], check=True,
                             capture_output=True, text=True).stdout.split()
        return dict(zip(("summed", "spoiled", "flags", "open", "waits_late", "asked_in_flight", "parity_wrong"),
                        map(int, out)))
    return run


ITEMS = [[32], [32, 32, 32], [1, 0, 5, 32, 8, 9, 0, 4, 31], [0, 0, 3], [4, 4, 4, 4], [12, 7, 32]]


def batches(lives):
    return sum(-(-n // 4) for n in lives)


@pytest.mark.parametrize("lives", ITEMS)
def test_every_row_is_summed_once_where_all_copies_arrive(walk, lives):
    r = walk(-1, 0, lives)
    assert r == {"summed": sum(lives), "spoiled": 0, "flags": 0, "open": 0, "waits_late": 0, "asked_in_flight": 0,
                 "parity_wrong": 0}


@pytest.mark.parametrize("lives", ITEMS)
def test_a_copy_that_does_not_arrive_ends_the_sums_cleanly(walk, lives):
    """For each batch in turn: no row is summed from its wait on, nothing more is asked for or waited
    for, and every other copy has been waited for at the end; the late one, too, where it comes in that time."""
    order = []  # batches in the order in which the walk asks for them: item, rows before it
    for q, n in enumerate(lives):
        order += [(q, r) for r in range(0, n, 4)]
    before = [sum(lives[:q]) + r for q, r in order]
    for late in range(batches(lives)):
        for arrives_at in (0, 2):
            r = walk(late, arrives_at, lives)
            assert r["summed"] == before[late] and r["spoiled"] == sum(lives) - before[late]
            assert r["flags"] == 1 and r["waits_late"] == 2
            assert r["open"] == (0 if arrives_at else 1)
            assert not r["asked_in_flight"] and not r["parity_wrong"]
