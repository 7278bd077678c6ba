"""The tile kernel's P barriers under every interleaving of its warps (CPU).

The four softmax warps of a row tile write P(j) in two halves and arrive on a
barrier for each; the issuing warp waits for them before the products that read
P.  An mbarrier only counts arrivals, so a warp that runs ahead could complete
a phase in place of one that lags.  The model walks all states of the protocol
with the kernel's own choice of barriers (chunk_schedule.h); the tensor core is
infinitely fast in it, which is the least order that the kernel can rely on.
"""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILES, WARPS = 5, 3  # (a third warp adds the states in which two run ahead of one)


@pytest.fixture(scope="module")
def barriers(tmp_path_factory):
    """(nq, half, tile) -> (slot, parity) of row tile 0, from the header."""
    d = tmp_path_factory.mktemp("schedule")
    src = d / "schedule.cpp"
    src.write_text("""#include <cstdio>
#include "chunk_schedule.h"
int main() {
  for (int nq = 1; nq <= 2; ++nq)
    for (int h = 0; h < 2; ++h)
      for (int j = 0; j < %d; ++j) {
        const fp8kv::BarrierAt b = fp8kv::p_ready_at(nq, 0, h, j);
        std::printf("%%d %%d %%d %%d %%d\\n", nq, h, j, b.slot, b.parity);
      }
}
""" % TILES)
    exe = d / "schedule"
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "fp8_e4m3_paged_gb300", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return {(nq, h, j): (slot, parity) for nq, h, j, slot, parity in
            (tuple(map(int, line.split())) for line in out.splitlines())}


def programs(nq):
    """Steps of the issuing warp and of the others."""
    issuer, other = [("qk", 0)], []
    for j in range(TILES):
        other += [("see", j), ("arrive", 0, j), ("arrive", 1, j)]
        more = [("qk", j + 1)] if j + 1 < TILES else []
        if nq == 1:  # QK(j+1) between the halves of PV(j)
            issuer += [("see", j), ("arrive", 0, j), ("wait", 0, j), ("arrive", 1, j)] + more + [("wait", 1, j)]
        else:
            issuer += [("see", j), ("arrive", 0, j), ("arrive", 1, j), ("wait", 0, j), ("wait", 1, j)] + more
    return [tuple(issuer)] + [tuple(other)] * (WARPS - 1)


def walk(nq, at):
    """A state in which the issuer passes a wait although some warp has not arrived, or that nothing leaves; None if
    there is none."""
    steps = programs(nq)
    keys = sorted({(h, at[nq, h, j][0]) for h in range(2) for j in range(TILES)})
    # state: place of each warp, then (phase, arrivals) of each barrier; S(j) is there once the issuer is past qk(j)
    start = ((0,) * WARPS, ((0, 0),) * len(keys))
    qk_at = {step[1]: i for i, step in enumerate(steps[0]) if step[0] == "qk"}
    arrive_at = [{step[1:]: i for i, step in enumerate(p) if step[0] == "arrive"} for p in steps]
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        place, bars = state
        moved = False
        for w in range(WARPS):
            if place[w] == len(steps[w]):
                continue
            step = steps[w][place[w]]
            new = bars
            if step[0] == "see" and place[0] <= qk_at[step[1]]:
                continue
            if step[0] == "arrive":
                i = keys.index((step[1], at[(nq,) + step[1:]][0]))
                phase, n = bars[i]
                new = bars[:i] + (((phase + 1, 0) if n + 1 == WARPS else (phase, n + 1)),) + bars[i + 1:]
            if step[0] == "wait":
                slot, parity = at[(nq,) + step[1:]]
                if bars[keys.index((step[1], slot))][0] & 1 == parity:  # that phase is not complete
                    continue
                if any(place[x] <= arrive_at[x][step[1:]] for x in range(WARPS)):
                    return "passed early", step, place
            moved = True
            nxt = (place[:w] + (place[w] + 1,) + place[w + 1:], new)
            if nxt not in seen:
                seen.add(nxt)
                todo.append(nxt)
        if not moved and any(place[w] < len(steps[w]) for w in range(WARPS)):
            return "stuck", place
    return None


@pytest.mark.parametrize("nq", [1, 2])
def test_no_warp_arrives_in_place_of_another(barriers, nq):
    assert walk(nq, barriers) is None


def test_the_walk_finds_a_shared_barrier(barriers):
    """One barrier for the second half of every tile, planted in the model: a fast warp stands in for a slow one."""
    one = {key: (0, key[2] & 1) for key in barriers}
    assert walk(1, one)[0] == "passed early"
    assert walk(2, one) is None
