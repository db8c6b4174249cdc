"""Prompts, rotation and attention write nothing outside their buffers (canaries on both sides of each,
of the workspaces too), and give the same bits with programmatic dependent launch on and off, in chains
of calls that each read what the one before wrote."""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402
import test_attend_gpu  # noqa: E402
import test_prompts_gpu  # noqa: E402
import test_rotate_gpu  # noqa: E402
from test_guards_gpu import Guarded  # noqa: E402


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# whole prompts with empty ones, a cut prompt, CTAs that share prompts, token by token
PROMPTS = {"whole": dict(lens=[1, 0, 129, 64], H=3), "cut": dict(lens=[1500, 37], H=2),
           "shared": dict(lens=[600 + (131 * i) % 401 for i in range(40)], H=8),
           "bf16": dict(lens=[700, 130], H=4, N=64, state=torch.bfloat16),
           "by token": dict(lens=[20, 150], H=3, P=24)}


def prompts_arguments(op, d, guard):
    g = test_prompts_gpu.to_gpu(d)
    out = torch.full(g["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    n = op.prompts_workspace_bytes(g["pool"], g["x"], g["B"], g["slots"])
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    if guard:
        guards = [Guarded(t) for t in (g["pool"], out, ws)]
        g["pool"], out, ws = (t.t for t in guards)
    else:
        guards = []
    args = [g[k] for k in ("pool", "slots", "cu", "x", "dt", "dt_bias", "A", "B", "C", "D")]
    return [*args, out, ws], g["fresh"], guards


@pytest.mark.parametrize("kind", PROMPTS)
def test_prompts_stay_in_their_buffers(op, kind):
    d = test_prompts_gpu.make(seed=51, extra=0, **PROMPTS[kind])  # every slot is named
    d["slots"][0] = d["pool"].shape[0]  # one prompt is skipped
    args, fresh, _ = prompts_arguments(op, d, False)
    op.prompts(*args, fresh=fresh)
    mine, fresh, guards = prompts_arguments(op, d, True)
    op.prompts(*mine, fresh=fresh)
    assert op.get_error() == (2, 0)
    assert all(g.intact() for g in guards)
    assert same(mine[0], args[0]) and same(mine[10], args[10])


@pytest.mark.parametrize("kind", PROMPTS)
def test_prompts_without_dependent_launch(op, kind):
    d = test_prompts_gpu.make(seed=52, **PROMPTS[kind])
    results = []
    try:
        for pdl in (True, False):
            ssu.ssu_set_pdl(op.handle, pdl)
            args, fresh, _ = prompts_arguments(op, d, False)
            for i in range(6):  # each continues from the slots of the one before
                args[3].mul_(0.96875)
                op.prompts(*args, fresh=fresh if i == 0 else None)
                op.prompts(*args)
            torch.cuda.synchronize()
            results.append((args[0], args[10]))
    finally:
        ssu.ssu_set_pdl(op.handle, True)
    assert same(results[0][0], results[1][0]) and same(results[0][1], results[1][1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rotation_stays_in_its_buffers(op, D):
    d = test_rotate_gpu.make(61, 5, 2, D, 32, seed=53)
    cells = d["k_pages"].shape[0] * d["k_pages"].shape[1]
    # the first and the last row of the cache, one token not stored, one skipped
    slots = torch.randperm(cells - 2)[:61] + 1
    slots[:4] = torch.tensor([0, cells - 1, -1, cells])
    d["slots"] = slots.to(d["slots"].dtype).cuda()
    ref = {k: v.clone() for k, v in d.items()}
    op.rotate_qk(**ref)
    guards = {k: Guarded(d[k]) for k in ("q_out", "k_pages", "v_pages")}
    op.rotate_qk(**{**d, **{k: g.t for k, g in guards.items()}})
    assert op.get_error() == (2, 3)
    for k, g in guards.items():
        assert g.intact() and same(g.t, ref[k])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[0, 1, 700, 33], [9000], [(37 * i) % 301 for i in range(300)]],
                         ids=["few", "long", "many"])
def test_attention_stays_in_its_buffers(op, D, lens):
    d = test_attend_gpu.make(lens, Hq=8, Hk=2, D=D, seed=54)
    ref = {k: v.clone() for k, v in d.items()}
    op.attend(**ref, workspace=test_attend_gpu.workspace(op, d))
    n = op.attend_workspace_bytes(d["q"], d["k_pages"])
    out, ws = Guarded(d["out"]), Guarded(torch.zeros(n, dtype=torch.uint8, device="cuda"))
    for _ in range(2):
        op.attend(**{**d, "out": out.t}, workspace=ws.t)
        assert out.intact() and ws.intact() and same(out.t, ref["out"])
    assert op.get_error() == (0, -1)


@pytest.mark.parametrize("D", [64, 128])
def test_tokens_without_dependent_launch(op, D):
    """Rotation into the cache and attention over it, whose output is the next token's query."""
    results = []
    try:
        for pdl in (True, False):
            ssu.ssu_set_pdl(op.handle, pdl)
            lens = [0, 5, 900, 63]
            a = test_attend_gpu.make([n + 20 for n in lens], Hq=8, Hk=2, D=D, seed=55)
            r = test_rotate_gpu.make(len(lens), 8, 2, D, 32, places=2000, seed=56)
            a["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
            ws = torch.zeros(op.attend_workspace_bytes(a["q"], a["k_pages"]), dtype=torch.uint8,
                             device="cuda")
            who = torch.arange(len(lens), device="cuda")
            outs = []
            q = r["q"]
            for _ in range(16):
                at = a["lengths"].long()
                slots = (a["page_table"][who, at // 16] * 16 + at % 16).int()
                op.rotate_qk(q, r["k"], r["v"], r["q_weight"], r["k_weight"], r["table"],
                             a["lengths"].clone(), a["q"], a["k_pages"], a["v_pages"], slots)
                a["lengths"] += 1
                op.attend(**a, workspace=ws)
                outs.append(a["out"].clone())
                q = outs[-1]
            torch.cuda.synchronize()
            results.append(torch.stack(outs))
    finally:
        ssu.ssu_set_pdl(op.handle, True)
    assert same(*results) and results[0].isfinite().all()
    assert op.get_error() == (0, -1)


def test_a_head_without_a_finite_score(op):
    """Scores of minus infinity alone: zeros, as for an empty cache; the other heads are as they are."""
    d = test_attend_gpu.make([40, 300], Hq=4, Hk=2, D=64, seed=57)
    op.attend(**d, workspace=test_attend_gpu.workspace(op, d))
    want = d["out"].clone()
    d["q"][:, :2] = 1.0
    d["k_pages"][:, :, 0] = float("-inf")
    op.attend(**d, workspace=test_attend_gpu.workspace(op, d))
    torch.cuda.synchronize()
    assert (d["out"][:, :2] == 0).all() and torch.equal(d["out"][:, 2:], want[:, 2:])
