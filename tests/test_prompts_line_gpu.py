"""Prompts whose chunks CTAs share, so that states are handed from CTA to CTA: the same bits from call
to call, eagerly and in a graph."""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402
from test_prompts_gpu import check, make, reference, to_gpu  # noqa: E402


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def shared(seed, state=torch.float32):
    """40 prompts, four pairs of columns each: 160 CTAs' work on 152 SMs or so."""
    return make([600 + (131 * i) % 401 for i in range(40)], H=8, state=state, seed=seed)


def arguments(op, d):
    g = to_gpu(d)
    out = torch.full(g["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    n = op.prompts_workspace_bytes(g["pool"], g["x"], g["B"], g["slots"])
    assert n > 0
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    args = [g[k] for k in ("pool", "slots", "cu", "x", "dt", "dt_bias", "A", "B", "C", "D")]
    return g, out, [*args, out, ws]


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_handed_on_states_are_whole(op, state):
    d = shared(1, state)
    ref = reference(d)
    g, out, args = arguments(op, d)
    start = g["pool"].clone()
    first = None
    for _ in range(40):
        g["pool"].copy_(start)
        out.fill_(7.0)
        op.prompts(*args, fresh=g["fresh"])
        if first is None:
            first = out.clone(), g["pool"].clone()
            check(d, out.cpu(), g["pool"].cpu(), ref)
        assert torch.equal(out, first[0]) and torch.equal(g["pool"], first[1])
    assert op.get_error() == (0, -1)


def test_in_a_graph(op):
    d = shared(2)
    ref = reference(d)
    g, out, args = arguments(op, d)
    start = g["pool"].clone()
    op.prompts(*args, fresh=g["fresh"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.prompts(*args, fresh=g["fresh"])
    for _ in range(3):
        g["pool"].copy_(start)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(d, out.cpu(), g["pool"].cpu(), ref)
