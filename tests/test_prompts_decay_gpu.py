"""A decay that is not a number shows: A or a token's dt of NaN makes the head's readouts and state NaN
from that token on, as in the recurrence, and leaves everything else as it would be without it."""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402
from test_prompts_gpu import call, check, make, reference  # noqa: E402

NAN, INF = float("nan"), float("inf")
# whole prompts in chunks, a cut prompt, CTAs that share prompts, token by token
LENS = [([1, 37, 300], 64), ([1500], 64), ([600 + (131 * i) % 401 for i in range(40)], 64),
        ([5, 150], 24)]


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


@pytest.mark.parametrize("lens,P", LENS, ids=["whole", "cut", "shared", "by token"])
def test_a_is_nan(op, lens, P):
    d = make(lens, H=8 if len(lens) > 3 else 3, P=P, seed=41)
    clean = call(op, d)
    d["A"][1] = NAN
    out, pool = call(op, d)
    slots = d["slots"].long()
    assert out[:, 1].isnan().all() and pool[slots, 1].isnan().all()
    others = [h for h in range(d["A"].shape[0]) if h != 1]
    assert torch.equal(out[:, others], clean[0][:, others])
    assert torch.equal(pool[:, others], clean[1][:, others])
    # the reference agrees about what is NaN
    few = make([3], H=3, P=P, seed=42)
    few["A"][1] = NAN
    y, state, _, _ = reference(few)
    assert y[:, 1].isnan().all() and state[few["slots"].long(), 1].isnan().all()


@pytest.mark.parametrize("lens,P", LENS, ids=["whole", "cut", "shared", "by token"])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_tokens_dt(op, lens, P, bad):
    """dt = +inf takes the state away and leaves infinities or NaN of its own."""
    d = make(lens, H=8 if len(lens) > 3 else 3, P=P, seed=43)
    clean = call(op, d)
    lo, hi = d["cu"][-2].item(), d["cu"][-1].item()
    for t in (lo, lo + 2, (lo + hi) // 2, hi - 1):
        dt = d["dt"][t, 1].clone()
        d["dt"][t, 1] = bad
        out, pool = call(op, d)
        keep = torch.ones_like(out, dtype=torch.bool)
        keep[t:hi, 1] = False
        assert torch.equal(out[keep], clean[0][keep])
        if bad != bad:
            assert out[~keep].isnan().all() and pool[d["slots"][-1].item(), 1].isnan().all()
        else:
            assert not out[t, 1].isfinite().any()
        d["dt"][t, 1] = dt


@pytest.mark.parametrize("lens,P", LENS[:2] + LENS[3:], ids=["whole", "cut", "by token"])
def test_a_is_minus_infinity(op, lens, P):
    """exp(dt A) is 0: every token starts anew."""
    d = make(lens, H=3, P=P, seed=44)
    d["A"][1] = -INF
    check(d, *call(op, d), reference(d))
