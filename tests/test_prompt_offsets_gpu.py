"""Prompts whose offsets run backwards, so that good ones among them overlap: those after the first
are skipped and counted, the rest is right, and nothing outside the call's buffers is written (a
canary lies on each side of the workspace, which has room for prompts that do not overlap)."""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402
from test_prompts_gpu import check, make, reference, to_gpu  # noqa: E402

GUARD, CANARY = 1 << 20, 0xA5


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def guarded_call(op, d):
    g = to_gpu(d)
    out = torch.full(g["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    n = op.prompts_workspace_bytes(g["pool"], g["x"], g["B"], g["slots"])
    room = torch.full((n + 2 * GUARD,), CANARY, dtype=torch.uint8, device="cuda")
    op.prompts(g["pool"], g["slots"], g["cu"], g["x"], g["dt"], g["dt_bias"], g["A"], g["B"],
               g["C"], g["D"], out, room[GUARD:GUARD + n], fresh=g["fresh"])
    torch.cuda.synchronize()
    assert (room[:GUARD] == CANARY).all() and (room[GUARD + n:] == CANARY).all()
    return out.cpu(), g["pool"].cpu(), n


@pytest.mark.parametrize("idx", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("N", [64, 128])
def test_two_prompts_over_the_same_rows(op, N, idx):
    """Cut into stretches, each of the two would take all of the workspace."""
    T = 12800
    d = make([T, 0, 0], H=2, N=N, seed=1, idx=idx)
    d["cu"] = torch.tensor([0, T, 0, T], dtype=idx)  # prompt 1 runs backwards
    op.get_error()
    out, pool, n = guarded_call(op, d)
    assert n > 0
    check(d, out, pool, reference(d, skip=(1, 2)))
    assert op.get_error() == (2, 1)


def test_overlaps_in_part_and_empty_prompts_in_between(op):
    d = make([0] * 6, H=2, seed=2, gap=1500)
    #                       0    1    2     3     4          5
    d["cu"] = torch.tensor([300, 900, 900, 500, 500, 200, 1500], dtype=torch.int32)
    # 2 and 4 run backwards; 3 is empty inside prompt 0; 5 shares rows with prompt 0
    d["fresh"][3] = True
    op.get_error()
    out, pool, _ = guarded_call(op, d)
    check(d, out, pool, reference(d, skip=(2, 4, 5)))
    assert op.get_error() == (3, 2)


def test_a_bad_prompt_is_in_nobodys_way(op):
    """A prompt that is skipped for its end or its slot keeps its rows from nobody."""
    d = make([0] * 5, H=2, seed=3, gap=900)
    d["cu"] = torch.tensor([100, 5000, 50, 400, 100, 900], dtype=torch.int32)
    # 0 ends outside the rows, 1 and 3 run backwards, 2 is good but has no slot, 4 is good
    d["slots"][2] = -1
    op.get_error()
    out, pool, _ = guarded_call(op, d)
    check(d, out, pool, reference(d, skip=(0, 1, 2, 3)))
    assert op.get_error() == (4, 0)


def test_overlaps_among_prompts_that_share_ctas(op):
    lens = [500 + (97 * i) % 301 for i in range(39)]
    lens[20] = 3100
    d = make(lens, H=8, seed=4)
    d["cu"][31] = 0  # prompt 30 runs backwards, prompt 31 covers all the rows before its own
    ref = reference(d, skip=(30, 31))
    op.get_error()
    out, pool, n = guarded_call(op, d)
    assert n > 0
    check(d, out, pool, ref)
    assert op.get_error() == (2, 30)


def clean_call(op, d, skip):
    """The same prompts at offsets that do not run backwards, those of ``skip`` without a slot."""
    slots = d["slots"].clone()
    slots[list(skip)] = -1
    out, pool, _ = guarded_call(op, {**d, "slots": slots})
    assert op.get_error() == (len(skip), min(skip))
    return out, pool


@pytest.mark.parametrize("lens,H", [
    ([3 + i % 5 for i in range(800)], 2),                  # whole prompts
    ([3 + i % 5 for i in range(799)] + [3000], 2),         # the last one cut
    ([800 + 13 * (i % 9) if i != 10 else 5000 for i in range(360)], 2)],  # shared, and one cut
    ids=["whole", "cut", "shared"])
def test_more_prompts_than_a_scan_takes_at_once(op, lens, H):
    d = make(lens, H=H, seed=5)
    n = len(lens)
    bad = [(n // 7, 0), (n * 5 // 8, n // 3), (n * 7 // 8, n * 3 // 8)]
    skip = {p - 1 for p, _ in bad} | {p for p, _ in bad}
    op.get_error()
    want = clean_call(op, d, sorted(skip))
    cu = d["cu"].clone()
    for p, to in bad:  # prompt p - 1 runs back to the start of another, prompt p from there on
        d["cu"][p] = cu[to]
    out, pool, _ = guarded_call(op, d)
    assert op.get_error() == (len(skip), min(skip))
    assert torch.equal(out, want[0]) and torch.equal(pool, want[1])
