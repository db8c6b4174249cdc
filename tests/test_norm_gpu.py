"""The residual addition with RMS norm (``ssu_add_norm``) against its formula in fp64.

Tolerances, derived before any run: the sum x + residual is rounded once to fp32 (2^-24 |r|), the
mean of its squares is a sum of at most 32 + 16 + 5 roundings deep (2^-19 of it, half of that of its
root), and the three products add 2^-22: y is within 2^-18 |y| + 2^-23 rms of the formula's (an r
that cancels keeps the error of its sum), before its rounding to bf16 (2^-8) or e4m3.  A residual
is within half a step of the sum.  A scale is within 2^-18 of the largest |y| of its group over
448; an e4m3 value q stands for y / scale: within half a step, 2^-4 |y / scale|, or half the
smallest step, 2^-10, and those 2^-17 of it.
"""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402
from test_guards_gpu import Guarded  # noqa: E402


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def make(T, W, residual, e4m3=False, group=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T + W)
    d = dict(x=torch.randn(T, W, generator=g, device="cuda").bfloat16(), residual=None, scales=None,
             weight=torch.rand(W, generator=g, device="cuda") + 0.5,
             out=torch.zeros(T, W, device="cuda").to(torch.float8_e4m3fn if e4m3
                                                     else torch.bfloat16))
    if residual is not None:
        d["residual"] = (4 * torch.randn(T, W, generator=g, device="cuda")).to(residual)
    if e4m3:
        d["scales"] = torch.zeros(T, W // (group or W), device="cuda")
    return d


def formula(d, eps=1e-6):
    r = d["x"].double()
    if d["residual"] is not None:
        r = r + d["residual"].double()
    rms = torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    return r, r / rms * d["weight"].double(), d["weight"].double() * 2.0 ** -23


def run(op, d, **kw):
    residual = d["residual"].clone() if d["residual"] is not None else None
    op.add_norm(d["x"], d["weight"], d["out"], residual=residual, scales=d["scales"], **kw)
    torch.cuda.synchronize()
    return residual


def check(d, residual, want):
    r, y, slack = want
    if residual is not None:
        half = 2.0 ** -8 if residual.dtype == torch.bfloat16 else 2.0 ** -24
        assert ((residual.double() - r).abs() <= half * r.abs() + 2.0 ** -23 * r.abs()).all()
    if d["scales"] is None:
        assert ((d["out"].double() - y).abs() <= (2.0 ** -8 + 2.0 ** -17) * y.abs() + slack).all()
        return
    parts = y.view(len(y), d["scales"].shape[1], -1)
    scale = (parts.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    assert ((d["scales"].double() - scale).abs() <= 2.0 ** -17 * scale).all()
    units = (parts / d["scales"].double()[..., None]).view_as(y)
    slack = (slack.expand_as(y).reshape_as(parts) / d["scales"].double()[..., None]).view_as(y)
    err = (d["out"].float().double() - units).abs()
    assert (err <= torch.maximum(2.0 ** -4 * units.abs(), torch.full_like(err, 2.0 ** -10)) +
            2.0 ** -17 * units.abs() + slack).all()
    assert (d["out"].float().abs().view_as(parts).amax(-1) >= 416).all()  # scales are used fully


SIZES = [(1, 8), (3, 64), (5, 72), (8, 4096), (130, 256), (7, 1000), (2, 4104), (9, 8192),
         (1, 16384), (2, 20000), (3, 32768), (777, 2560)]


@pytest.mark.parametrize("T,W", SIZES, ids=str)
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32],
                         ids=["none", "bf16", "f32"])
def test_bf16(op, T, W, residual):
    d = make(T, W, residual)
    check(d, run(op, d), formula(d))


@pytest.mark.parametrize("T,W,group", [
    (1, 32, 32), (3, 64, 64), (5, 72, 72), (8, 4096, 128), (130, 256, 256), (7, 1000, 1000),
    (2, 4096, 32), (9, 8192, 64), (1, 16384, 256), (2, 20000, 32), (3, 32768, 128),
    (777, 2560, 2560), (33, 384, 128), (4, 8, 8)], ids=str)
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32],
                         ids=["none", "bf16", "f32"])
def test_e4m3(op, T, W, group, residual):
    d = make(T, W, residual, True, group)
    check(d, run(op, d), formula(d))


@pytest.mark.parametrize("e4m3", [False, True])
def test_strides_and_rows_between(op, e4m3):
    T, W, group = 70, 512, 64
    d = make(T, W, torch.float32, e4m3, group)
    big = {k: torch.zeros(2 * T, W + 24, device="cuda").to(d[k].dtype)
           for k in ("x", "residual", "out")}
    view = {k: t[::2, 8:8 + W] for k, t in big.items()}
    for k in ("x", "residual"):
        view[k].copy_(d[k])
    scales = torch.zeros(W // group, 3 * T, device="cuda") if e4m3 else None
    op.add_norm(view["x"], d["weight"], view["out"], residual=view["residual"],
                scales=scales[:, ::3].t() if e4m3 else None)
    torch.cuda.synchronize()
    e = dict(d, out=view["out"].contiguous(), scales=scales[:, ::3].t().contiguous() if e4m3
             else None)
    check(e, view["residual"].contiguous(), formula(d))
    for k in ("residual", "out"):
        assert (big[k][1::2].float() == 0).all()
        assert (big[k][:, :8].float() == 0).all() and (big[k][:, 8 + W:].float() == 0).all()
    if e4m3:
        assert (scales[:, 1::3] == 0).all() and (scales[:, 2::3] == 0).all()


def test_out_may_be_x_and_x_may_repeat(op):
    d = make(20, 768, torch.bfloat16)
    want = formula(d)
    one = dict(d, x=d["x"][:1].expand(20, -1))  # one row for every token: stride 0
    check(one, run(op, one), formula(one))
    d["out"] = d["x"]
    check(d, run(op, d), want)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_bad_values_stay_in_their_token(op, e4m3, bad):
    d = make(9, 1024, torch.float32, e4m3, 128)
    clean = {k: v.clone() for k, v in d.items() if v is not None}
    r0 = run(op, dict(d, out=clean["out"], scales=clean.get("scales")))
    d["x"][4, 300] = bad
    r = run(op, d)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    assert torch.equal(r[keep], r0[keep])
    assert torch.equal(d["out"].float()[keep], clean["out"].float()[keep])
    got = d["out"].float()[4]
    if e4m3:
        assert torch.equal(d["scales"][keep], clean["scales"][keep])
        assert torch.isnan(d["scales"][4, 300 // 128])
        got = got * d["scales"][4].repeat_interleave(128)
    assert torch.isnan(got[300])
    if bad == bad:  # an infinite length: what is finite becomes zero
        assert (got[[0, 1023]] == 0).all()
    else:
        assert torch.isnan(got).all()


@pytest.mark.parametrize("fill", [0.0, 1e-30, 3e38])
def test_extreme_rows(op, fill):
    """Rows of zeros, of what squares to nothing, and of what squares to infinity (which is zero)."""
    d = make(3, 256, None, True, 128)
    d["x"].fill_(fill)
    run(op, d)
    assert torch.isfinite(d["out"].float()).all() and torch.isfinite(d["scales"]).all()
    if fill != 1e-30:
        assert (d["out"].float() == 0).all() and (d["scales"] == 2.0 ** -126).all()
    else:
        y = d["x"].double() / 1e-3 * d["weight"].double()
        got = d["out"].float().double() * d["scales"].double().repeat_interleave(128, 1)
        assert ((got - y).abs() <= 2.0 ** -3 * y).all()


def test_zero_tokens_and_graphs(op):
    op.add_norm(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                torch.ones(64, device="cuda"),
                torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    d = make(50, 2048, torch.bfloat16, True, 128)
    start = d["residual"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.add_norm(d["x"], d["weight"], d["out"], residual=d["residual"], scales=d["scales"])
    for seed in range(2):
        e = make(50, 2048, torch.bfloat16, True, 128, seed=seed)
        d["x"].copy_(e["x"])
        d["residual"].copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        check(d, d["residual"], formula(dict(d, residual=start)))


@pytest.mark.parametrize("T,W,group", [(3, 72, 72), (700, 1024, 64), (5, 20000, 32)], ids=str)
def test_calls_stay_in_their_buffers(op, T, W, group):
    """Canaries on both sides of what a call writes."""
    for e4m3 in (False, True):
        d = make(T, W, torch.bfloat16, e4m3, group)
        r = run(op, d)
        guards = {"residual": Guarded(d["residual"]), "out": Guarded(torch.zeros_like(d["out"].view(
            torch.uint8) if e4m3 else d["out"]))}
        if e4m3:
            guards["scales"] = Guarded(torch.zeros_like(d["scales"]))
        out = guards["out"].t.view(torch.float8_e4m3fn) if e4m3 else guards["out"].t
        op.add_norm(d["x"], d["weight"], out, residual=guards["residual"].t,
                    scales=guards["scales"].t if e4m3 else None)
        torch.cuda.synchronize()
        assert all(g.intact() for g in guards.values())
        assert torch.equal(guards["residual"].t, r) and torch.equal(out.float(), d["out"].float())
        if e4m3:
            assert torch.equal(guards["scales"].t, d["scales"])


def test_rows_past_32_bits(op):
    """More than 2^31 elements: the last rows."""
    T, W = 2 ** 31 // 8192 + 40, 8192
    x = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, W, device="cuda").bfloat16()
    out = torch.empty(T, W, dtype=torch.float8_e4m3fn, device="cuda")
    d = dict(x=x[-3:], residual=None, weight=torch.rand(W, device="cuda") + 0.5, out=out[-3:],
             scales=torch.zeros(T, 1, device="cuda"))
    op.add_norm(x, d["weight"], out, scales=d["scales"])
    torch.cuda.synchronize()
    check(dict(d, scales=d["scales"][-3:]), None, formula(d))
    assert (out[::4096].view(torch.uint8)[:-1] == 0).all()
