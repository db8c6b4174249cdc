"""Where an infinity or NaN in one token's operands ends: the readouts and states that the recurrence
makes infinite or NaN, and no others.  Tolerances as in test_delta_gpu.py."""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402
from test_delta_gpu import call, make, reference, step  # noqa: E402


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def close_where_finite(got, want, tol):
    """Not finite exactly where the recurrence is not; elsewhere within `tol`."""
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), finite)
    assert ((got - want).abs() <= tol)[finite].all()


FORMS = {"one token": ([1, 1, 1], 128, 128), "few tokens": ([9, 6, 5], 128, 128),
         "few, dstate 64": ([9, 6, 5], 72, 64), "token by token, dstate 256": ([40, 60], 64, 256),
         "chunks": ([100, 150], 128, 128), "chunks, dstate 64": ([90, 80], 72, 64)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_readouts_and_states_are_bad_where_the_recurrence_is(op, form, bad, where):
    """One element of one token: a query's reaches its token's readouts of its heads, a key's also the
    states of its heads and what is read of them from then on, a value's one row of one head."""
    lens, P, N = FORMS[form]
    d = make(lens, P=P, N=N, seed=137)
    if max(lens) == 1:
        d["fresh"] = None
    t = d["cu"][1].item() + lens[1] // 2
    tolerances = reference(d)
    d[where] = d[where].clone()
    d[where][t, 0, 3] = bad
    y, want, _, _, _ = reference(d)
    _, _, Y, R, most = tolerances
    if max(lens) == 1:
        pool, out = d["pool"].clone(), torch.zeros_like(d["v"])
        step(op, d, pool, out)
        torch.cuda.synchronize()
    else:
        out, pool = call(op, d)
    close_where_finite(out.double(), y, 2.0 ** -8 * y.abs() + (2.0 ** -7 + 2.0 ** -13) * Y)
    n = min(sum(lens), 1.0 / (1.0 - most))
    close_where_finite(pool.double(), want, (n * 2.0 ** -20 * R)[..., None].expand_as(want))
    bad_heads = {"q": 2, "k": 2, "v": 1}[where]
    assert (~torch.isfinite(out[t]).all(-1)).sum() == bad_heads  # the case is what it says


@pytest.mark.parametrize("P,N,state", [(72, 64, torch.bfloat16), (192, 128, torch.float32)], ids=str)
@pytest.mark.parametrize("where", ["k", "v", "dt"])
def test_states_after_a_chunk_taken_token_by_token(op, P, N, state, where):
    """The state of the prompt with the bad token, where a CTA's rows are not all the head's and in
    two slabs: NaN where it reaches, as the recurrence leaves it in other heads and rows."""
    d = make([100, 150], P=P, N=N, state=state, seed=109)
    y, want, Y, R, most = reference(d)
    t = 170
    d[where] = d[where].clone()
    d[where][(t, 0, 3) if where == "v" else (t, 0)] = float("nan")
    out, pool = call(op, d)
    slot = d["slots"][1].item()
    reached = torch.zeros(pool.shape[1:3], dtype=torch.bool, device="cuda")  # [H, P]
    if where == "k":
        reached[:2] = True  # the heads of key head 0
    elif where == "dt":
        reached[0] = True
    else:
        reached[0, 3] = True
    assert torch.isnan(pool[slot][reached]).all()
    err = (pool[slot].double() - want[slot]).norm(dim=-1)
    half = 2.0 ** -8 * want[slot].norm(dim=-1) if state == torch.bfloat16 else 0.0
    tol = min(250, 1.0 / (1.0 - most)) * 2.0 ** -20 * R[slot] + half
    assert (err <= tol)[~reached].all()
