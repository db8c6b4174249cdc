"""Long prompts with slow decays against the recurrence in fp64: thousands of tokens are alive at a
time.

Tolerances.  The decay is the same for all tokens here, so what fp32 makes of exp(softplus(dt) A) is
wrong in the same direction every time: by 2^-22 of it (softplus and exp, 2^-23.5 each at most, and a
product), over n = min(tokens, 1 / (1 - a)) tokens alive n 2^-22 of what they leave.  In chunks T's
elements are good to 2^-17, u = T R: a correction is off by sums of 2^-17 T_jl R_l.  Where all keys
are the same and gates are one, T is 1 and about -1 beside it, R_l is v_l less the value before,
sqrt(2) |v|: 2^-17 sqrt(2) / sqrt(3) |v| in the mean square, and 64 of them add up on one key as
squares, 8 times as much: 2^-14.3 |v|, where the row's state is |v| long.  Other keys and gates
cancel less.  So
* states: rows n 2^-20 R_p as in test_delta_gpu.py, and in the 2-norm of a call n 2^-22 + 2^-14
* readouts: 2^-8 |y| (rounded once) and (2^-13 + n 2^-22) Y, Y the magnitudes; in the 2-norm of a call
  0.0024 (a rounding is uniform in half a step, at most 2^-8 / sqrt(3) = 0.00226 of |y| in the mean
  square) and n 2^-22.
A pool in bf16: 2^-8 |S| more, its own rounding.
"""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402
from test_delta_gpu import call, make, reference  # noqa: E402


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def check(d, out, pool, ref):
    y, want, Y, R, most = ref
    n = min(len(d["v"]), 1.0 / (1.0 - most))
    err = (out.double() - y).abs()
    tol = 2.0 ** -8 * y.abs() + (2.0 ** -13 + n * 2.0 ** -22) * Y
    assert (err <= tol).all(), f"readout off by {(err / tol).max():.3g} of its tolerance"
    rel = err.norm() / y.norm()
    assert rel <= 0.0024 + n * 2.0 ** -22, f"readout 2-norm {rel:.3g}"
    at = d["slots"].long()
    err = (pool.double() - want).abs()[at]
    if pool.dtype == torch.bfloat16:
        err = (err - 2.0 ** -8 * want[at].abs()).clamp_min(0.0)
    rel = err.norm() / want[at].norm()
    assert rel <= n * 2.0 ** -22 + 2.0 ** -14, f"state 2-norm {rel:.3g}"
    assert (err.norm(dim=-1) <= n * 2.0 ** -20 * R[at]).all()


@pytest.mark.parametrize("A", [-1.0, -0.02], ids=["50 alive", "thousands alive"])
@pytest.mark.parametrize("keys", ["silu", "same", "normal"])
@pytest.mark.parametrize("N", [64, 128])
def test_long_prompts_with_slow_decays(op, N, keys, A):
    d = make([4000, 1500], H=4, N=N, G=2, seed=139, keys=keys)
    d["dt"] = torch.full_like(d["dt"], -4.0)
    d["dt_bias"] = torch.zeros_like(d["dt_bias"])
    d["A"] = torch.full_like(d["A"], A)
    ref = reference(d)
    check(d, *call(op, d), ref)
    d["b"] = torch.full_like(d["b"], 6.0)  # gates near one: the corrections cancel most
    check(d, *call(op, d), reference(d))


def test_a_long_prompt_through_a_bf16_pool(op):
    d = make([4000, 1500], H=4, P=64, N=64, G=2, seed=149, state=torch.bfloat16)
    d["dt"] = torch.full_like(d["dt"], -4.0)
    d["A"] = torch.full_like(d["A"], -0.05)
    check(d, *call(op, d), reference(d))


@pytest.mark.parametrize("lens,P,N,G", [([150, 0, 33], 128, 128, 2), ([300, 65], 72, 64, 1),
                                        ([1000], 256, 128, 4), ([70] * 40, 64, 64, 2)], ids=str)
def test_readouts_are_rounded_once(op, lens, P, N, G):
    """In chunks as token by token: no rounding of weights or corrections shows beside the readout's."""
    d = make(lens, P=P, N=N, G=G, seed=151)
    y, _, Y, _, _ = reference(d)
    out, _ = call(op, d)
    assert ((out.double() - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -13 * Y).all()
    assert (out.double() - y).norm() <= 0.0024 * y.norm()
