"""Norm and rotation of queries and keys into the paged cache (``ssu_rotate_qk``) against the
definition in fp64.

Tolerance, derived before any run: the fp32 sum of D squares, its root and the products carry
less than (D / 8 + 16) 2^-24 <= 2^-18 of |u|, a turned element is a sum of two such products, so
with R = |u_i cos| + |u_j sin| an element is within 2^-8 |value| (its rounding to bf16's 8
significant bits) + 2^-17 R.  Values are moved as they are.
"""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def make(T, Hq, Hk, D, rotary, page=16, places=500, seed=0, idx=torch.int32):
    g = torch.Generator().manual_seed(seed)
    pages = -(-max(T, 1) // page) + 2
    qkv = torch.randn(T, (Hq + 2 * Hk) * D, generator=g).bfloat16().cuda()
    angle = torch.rand(places, rotary // 2, generator=g) * 6.28
    return dict(
        q=qkv[:, :Hq * D].view(T, Hq, D), k=qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D),
        v=qkv[:, (Hq + Hk) * D:].view(T, Hk, D),
        q_weight=torch.rand(D, generator=g).cuda() + 0.5,
        k_weight=torch.rand(D, generator=g).cuda() + 0.5,
        table=torch.cat([angle.cos(), angle.sin()], 1).cuda(),
        positions=torch.randint(0, places, (T,), generator=g).to(idx).cuda(),
        q_out=torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16).cuda(),
        k_pages=torch.randn(pages, page, Hk, D, generator=g).bfloat16().cuda(),
        v_pages=torch.randn(pages, page, Hk, D, generator=g).bfloat16().cuda(),
        slots=torch.randperm(pages * page, generator=g)[:T].to(idx).cuda())


def turned(t, weight, table, positions, interleaved, eps):
    t = t.double().cpu()
    u = t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps) * weight.double().cpu()
    half = table.shape[1] // 2
    row = table.double().cpu()[positions.long().cpu()]
    c, s = row[:, None, :half], row[:, None, half:]
    m = torch.arange(half)
    i, j = (2 * m, 2 * m + 1) if interleaved else (m, m + half)
    out, mag = u.clone(), u.abs()
    out[..., i], out[..., j] = u[..., i] * c - u[..., j] * s, u[..., j] * c + u[..., i] * s
    mag[..., i] = (u[..., i] * c).abs() + (u[..., j] * s).abs()
    mag[..., j] = (u[..., j] * c).abs() + (u[..., i] * s).abs()
    return out, mag


def run_and_check(op, d, interleaved=False, eps=1e-6, skipped=(), unstored=()):
    """The call on ``d``; tokens in ``skipped`` write nothing, those in ``unstored`` only q."""
    T = d["q"].shape[0]
    k0, v0 = d["k_pages"].cpu(), d["v_pages"].cpu()
    pos = d["positions"].clone()
    pos[list(skipped)] = 0
    want_q, mag_q = turned(d["q"], d["q_weight"], d["table"], pos, interleaved, eps)
    want_k, mag_k = turned(d["k"], d["k_weight"], d["table"], pos, interleaved, eps)
    v = d["v"].cpu()
    op.rotate_qk(**d, eps=eps, interleaved=interleaved)
    torch.cuda.synchronize()
    q, k, vp = d["q_out"].cpu(), d["k_pages"].cpu(), d["v_pages"].cpu()
    live = torch.ones(T, dtype=torch.bool)
    live[list(skipped)] = False
    assert (q[~live] == 7.0).all()
    err, tol = (q.double() - want_q).abs(), 2.0 ** -8 * want_q.abs() + 2.0 ** -17 * mag_q
    assert (err <= tol)[live].all(), (err / tol)[live].max()
    live[list(unstored)] = False
    page = d["k_pages"].shape[1]
    at = d["slots"].long().cpu()[live]
    got = k[at // page, at % page].double()
    err = (got - want_k[live]).abs()
    assert (err <= 2.0 ** -8 * want_k[live].abs() + 2.0 ** -17 * mag_k[live]).all()
    assert torch.equal(vp[at // page, at % page].view(torch.int16), v[live].view(torch.int16))
    k0[at // page, at % page] = k[at // page, at % page]
    v0[at // page, at % page] = vp[at // page, at % page]
    assert torch.equal(k0, k) and torch.equal(v0, vp), "a cache row of no token was written"


@pytest.mark.parametrize("D,rotary", [(64, 64), (64, 16), (64, 0), (128, 128), (128, 96),
                                      (128, 16), (256, 256), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (7, 16, 2), (33, 6, 3)])
def test_shapes(op, T, Hq, Hk, D, rotary, interleaved):
    run_and_check(op, make(T, Hq, Hk, D, rotary, seed=T + D + rotary), interleaved)


@pytest.mark.parametrize("T", [2, 129, 1000])
@pytest.mark.parametrize("idx", [torch.int32, torch.int64], ids=["i32", "i64"])
def test_tokens_and_index_types(op, T, idx):
    run_and_check(op, make(T, 8, 2, 128, 128, page=24, seed=T, idx=idx))


def test_large_and_small_heads(op):
    """Heads of zeros (eps keeps them zero), tiny and huge values."""
    d = make(6, 4, 2, 128, 128, seed=3)
    d["q"][0], d["k"][1] = 0.0, 0.0
    d["q"][2] *= 1e-12
    d["q"][3] *= 1e15
    d["k"][3] *= 1e15
    run_and_check(op, d, eps=1e-6)
    assert (d["q_out"][0] == 0).all()


def test_in_place(op):
    d = make(50, 4, 2, 64, 64, seed=4)
    e = {k: v.clone() for k, v in d.items()}
    op.rotate_qk(**d)
    e["q_out"] = e["q"]
    op.rotate_qk(**e)
    torch.cuda.synchronize()
    assert torch.equal(e["q"], d["q_out"]) and torch.equal(e["k_pages"], d["k_pages"])


def test_strided_pages_and_indices(op):
    d = make(20, 4, 2, 64, 32, seed=5)
    n, page = d["k_pages"].shape[:2]
    both = torch.randn(n, 2, page, 3, 80, device="cuda").bfloat16()  # keys and values side by side
    d["k_pages"], d["v_pages"] = both[:, 0, :, :2, :64], both[:, 1, :, 1:, 8:72]
    d["positions"] = d["positions"].repeat_interleave(3)[::3]
    d["slots"] = d["slots"].repeat_interleave(2)[::2]
    d["q_out"] = torch.full((20, 4, 72), 7.0, device="cuda").bfloat16()[..., 8:]
    run_and_check(op, d)


def test_padding_and_bad_tokens(op):
    d = make(12, 4, 2, 128, 64, seed=6)
    op.get_error()
    total = d["k_pages"].shape[0] * d["k_pages"].shape[1]
    d["slots"][[2, 5]] = -1
    d["slots"][7] = total
    d["slots"][8] = -2
    d["positions"][3] = d["table"].shape[0]
    d["positions"][4] = -1
    run_and_check(op, d, skipped=(3, 4, 7, 8), unstored=(2, 5))
    assert op.get_error() == (4, 3)


def test_no_tokens(op):
    run_and_check(op, make(0, 4, 2, 64, 64))


def test_refusals(op):
    d = make(5, 4, 2, 128, 128, seed=8)

    def attempt(error, **change):
        with pytest.raises(error):
            op.rotate_qk(**{**d, **change})

    attempt(TypeError, q=d["q"].float())
    attempt(TypeError, q_weight=d["q_weight"].bfloat16())
    attempt(TypeError, slots=d["slots"].long())
    attempt(ValueError, v=d["v"][:, :1])
    attempt(ValueError, positions=d["positions"][:-1])
    attempt(ValueError, k_pages=d["k_pages"][..., :64])
    attempt(ValueError, q_out=d["q_out"].cpu())
    attempt(ValueError, q=d["q"].transpose(0, 2).contiguous().transpose(0, 2))
    attempt(ssu.SsuError, table=d["table"][:, :120].contiguous())
    attempt(ssu.SsuError, eps=-1.0)
    attempt(ssu.SsuError, eps=float("nan"))
    odd = torch.zeros(5, 4, 129, device="cuda").bfloat16()[..., 1:]
    attempt(ssu.SsuError, q_out=odd)
    assert (d["q_out"] == 7.0).all() and op.get_error() == (0, -1)
