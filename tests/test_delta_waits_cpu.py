"""What orders the delta rule's second pass, read off its source: faults here show only now and then
on a GPU, or only after another failure."""

from __future__ import annotations

import re
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "selective_state_update_02_gb300" / "csrc"
SOURCE = (CSRC / "ssu_delta_mma.cuh").read_text()


def between(start: str, end: str) -> str:
    at = SOURCE.index(start)
    return SOURCE[at:SOURCE.index(end, at)]


def test_no_load_is_in_flight_when_its_accumulator_is_handed_over():
    """R T^T overwrites S K^T, and weighted U's third part lies over U: where a piece of R or of
    weighted U is handed over, the warp's loads of the pieces from there have all been waited for.
    Walks both pieces through the statements that load, wait and hand over."""
    for block, bar in ((between("// R = beta v -", "// U with its weights"), "bar_r"),
                       (between("// U with its weights", "const float whole"), "bar_w")):
        statement = re.compile(
            r"(if \(x == 0\) )?(fetch\(([^)]*)\)|tc_wait_ld\(\)|hand_over\(" + bar + r"[^)]*\))")
        loop = block.index("fetch(0);")
        end = block.index(f"hand_over({bar}")
        handed = 0
        in_flight = True  # fetch(0), before the loop
        for x in (0, 1):
            for guard, what, _ in statement.findall(block[loop + len("fetch(0);"):end + 200]):
                if guard and x != 0:
                    continue
                if what.startswith("fetch"):
                    in_flight = True
                elif what.startswith("tc_wait_ld"):
                    in_flight = False
                else:
                    assert not in_flight, f"{bar}: piece {x} handed over with a load in flight"
                    handed += 1
                    break
        assert handed == 2


def test_every_wait_of_the_passes_is_bounded():
    """After a wait has given up, warps may see different flags and take different ways through a
    chunk: no barrier but the CTA's own, which every warp comes to, may count on the others."""
    assert "bar.sync" not in SOURCE and "barrier.sync" not in SOURCE
    assert "mbar_wait(" not in SOURCE and "try_wait" not in SOURCE
    second = SOURCE[SOURCE.index("// ---- the second pass"):]
    # the CTA's barriers: before the roles part and after they meet again
    roles = second.index("if (warp == kDeltaLoader)")
    end = second.index("tc_fence_before();\n    if (__syncthreads_or")
    assert "__syncthreads" not in second[roles:end]


def test_warps_take_one_way_through_a_chunk():
    """A warp's lanes agree on whether a chunk goes token by token: what follows are instructions of
    the whole warp."""
    for use in re.findall(r"[^\n]*flag\(\)[^\n]*", SOURCE):
        assert ("__any_sync" in use or "auto flag" in use or "!flag() && tok" in use  # one lane
                ), use
