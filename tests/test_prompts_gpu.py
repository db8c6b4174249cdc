"""Prompts (``ssu_update_prompts``) against the recurrence in fp64, token by token.

Tolerances, derived before any run.  With M the recurrence run on magnitudes (S <- dA S +
|dt x B|, from |S_0|) and Y = M |C| + |D x|, every form of the kernel stays within

* fp32 state: 2^-15 M.  A term that has passed n tokens carries at most n 2^-22 from the fp32
  dt, dA and products and a weight of at most exp(-a n), a = 0.0067 the least decay of these
  inputs: n exp(-a n) <= 55, so 2^-16.2; an operand split into two bf16 parts leaves 2^-18.
* bf16 state: 2^-8 M on top (one rounding at the end, of a value of at most M).
* readout: 2^-8 |y| (its own rounding: bf16 keeps 8 significant bits) + (2^-8 + 2^-14) Y:
  weights and states that enter a bf16 matrix product are rounded once, to 2^-8 of each term,
  and their fp32 errors are those of the state.  Over a whole call of random signs the errors
  add as squares, so the relative 2-norm stays within 2^-8 (a rounding is uniform between
  -2^-9 .. 2^-8 of its value, about 2^-9.2 in the mean square; two of them give 2^-8.7).
* everywhere 2^-126, below which fp32 has no full precision.
"""

from __future__ import annotations

import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402


TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def make(lens, H=4, P=64, N=128, G=1, state=torch.float32, seed=0, idx=torch.int32, extra=3,
         lead=0, gap=0):
    """Inputs of a call; ``lead`` rows before the first prompt and ``gap`` rows after the last are
    no prompt's."""
    g = torch.Generator().manual_seed(seed)
    bs, T = len(lens), lead + sum(lens) + gap
    cu = torch.tensor([lead] + [lead + s for s in itertools.accumulate(lens)])
    xbc = torch.randn(T, H * P + 2 * G * N, generator=g).bfloat16()
    d = dict(
        pool=torch.randn(bs + extra, H, P, N, generator=g).to(state),
        slots=torch.randperm(bs + extra, generator=g)[:bs].to(idx), cu=cu.to(idx),
        x=xbc[:, :H * P].view(T, H, P), B=xbc[:, H * P:H * P + G * N].view(T, G, N),
        C=xbc[:, H * P + G * N:].view(T, G, N),
        dt=(torch.rand(T, H, generator=g) * 4 - 4).bfloat16(),
        dt_bias=torch.rand(H, generator=g) * 2 - 1,
        A=-torch.exp(torch.rand(H, generator=g) * 2.77), D=torch.rand(H, generator=g),
        fresh=torch.rand(bs, generator=g) < 0.5)
    return d


def to_gpu(d):
    out = {}
    base = d["x"]._base
    if base is not None:  # keep x, B and C as views into one packed tensor
        gb = base.cuda()
        for k in ("x", "B", "C"):
            out[k] = gb.as_strided(d[k].shape, d[k].stride(), d[k].storage_offset())
    for k, v in d.items():
        if k not in out:
            out[k] = v.cuda()
    return out


def reference(d, skip=()):
    """The recurrence in fp64: (y, pool, Y, M) with the magnitudes of the tolerances; rows and
    slots that a call must not touch keep their start values (y: NaN)."""
    pool = d["pool"].double().clone()
    mag = torch.zeros_like(pool)
    y = torch.full(d["x"].shape, float("nan"), dtype=torch.float64)
    Y = torch.zeros(d["x"].shape, dtype=torch.float64)
    H, G = d["x"].shape[1], d["B"].shape[1]
    grp = torch.arange(H) // (H // G)
    dt = torch.nn.functional.softplus(d["dt"].double() + d["dt_bias"].double(), threshold=700)
    dA = torch.exp(dt * d["A"].double())
    x, B, C = (d[k].double() for k in ("x", "B", "C"))
    D = d["D"].double()[:, None]
    for b, slot in enumerate(d["slots"].tolist()):
        if b in skip:
            continue
        lo, hi = d["cu"][b].item(), d["cu"][b + 1].item()
        S = torch.zeros_like(pool[slot]) if d["fresh"] is not None and d["fresh"][b] \
            else pool[slot].clone()
        M = S.abs()
        for t in range(lo, hi):
            k = (x[t] * dt[t][:, None])[..., None] * B[t][grp][:, None]
            S = S * dA[t][:, None, None] + k
            M = M * dA[t][:, None, None] + k.abs()
            c = C[t][grp][..., None]
            y[t] = (S @ c)[..., 0] + D * x[t]
            Y[t] = (M @ c.abs())[..., 0] + (D * x[t]).abs()
        pool[slot], mag[slot] = S, M
    return y, pool, Y, mag


def call(op, d, fresh=True, **kw):
    g = to_gpu(d)
    out = torch.full(g["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((op.prompts_workspace_bytes(g["pool"], g["x"], g["B"], g["slots"]),), 0xff,
                    dtype=torch.uint8, device="cuda")
    op.prompts(g["pool"], g["slots"], g["cu"], g["x"], g["dt"], g["dt_bias"], g["A"], g["B"],
               g["C"], g["D"], out, ws, fresh=g["fresh"] if fresh else None, **kw)
    torch.cuda.synchronize()
    return out.cpu(), g["pool"].cpu()


def check(d, out, pool, ref):
    y, state, Y, M = ref
    run = ~torch.isnan(y)
    assert (out[~run] == 7.0).all(), "rows of no prompt were written"
    err = (out.double() - y).abs()[run]
    tol = (2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -14) * Y + TINY)[run]
    assert (err <= tol).all(), f"readout off by {(err / tol).max():.3g} of its tolerance"
    if run.sum() >= 4096:
        rel = err.norm() / y[run].norm()
        assert rel <= 2.0 ** -8, f"readout 2-norm {rel:.3g}"
    bf16 = pool.dtype == torch.bfloat16
    err = (pool.double() - state).abs()
    tol = M * (2.0 ** -15 + (2.0 ** -8 if bf16 else 0.0)) + TINY
    assert (err <= tol).all(), f"state off by {(err / tol.clamp_min(1e-300)).max():.3g} of its tolerance"


LENS = [
    [1], [2], [31], [37], [64], [127], [128], [129], [300], [1000],
    [1, 0, 5, 128, 129, 0, 77], [256, 3, 400], [16] * 40,
]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [64, 128])
def test_lengths(op, lens, N, state):
    d = make(lens, H=2, N=N, state=state, seed=len(lens) + sum(lens))
    check(d, *call(op, d), reference(d))


@pytest.mark.parametrize("H,P,N,G", [
    (8, 64, 128, 8), (6, 64, 128, 2), (4, 128, 128, 1), (3, 64, 256, 1), (2, 80, 128, 1),
    (5, 3, 64, 1), (2, 192, 64, 2), (1, 1, 128, 1), (4, 64, 64, 4), (2, 72, 256, 2),
    (16, 64, 128, 1)], ids=str)
@pytest.mark.parametrize("idx", [torch.int32, torch.int64], ids=["i32", "i64"])
def test_shapes(op, H, P, N, G, idx):
    d = make([150, 0, 33], H, P, N, G, seed=H * P + N, idx=idx)
    check(d, *call(op, d), reference(d))


def test_one_long_prompt_of_few_heads(op):
    """One prompt that is long for its heads: its chunks are spread over the device."""
    d = make([5003], H=2, seed=5)
    check(d, *call(op, d), reference(d))


def test_long_and_short_prompts(op):
    d = make([1, 2500, 3, 130, 900, 0, 64], H=4, G=2, seed=6)
    check(d, *call(op, d), reference(d))


@pytest.mark.parametrize("kind", ["strong", "none", "weak"])
@pytest.mark.parametrize("N", [64, 128])
def test_decays(op, kind, N):
    """dA that underflows to 0, dA that is exactly 1 (dt = 0 after softplus), and slow decays."""
    d = make([400, 129], H=4, N=N, seed=7)
    if kind == "strong":
        d["dt"] = torch.where(torch.rand(d["dt"].shape, generator=torch.Generator().manual_seed(1))
                              < 0.3, 60.0, 2.0).bfloat16()
        d["A"] = torch.tensor([-16.0, -8.0, -2.0, -0.5])
    elif kind == "none":
        d["dt"] = torch.full_like(d["dt"], -200.0)
    else:
        d["dt"] = torch.full_like(d["dt"], -4.0)
        d["A"] = -torch.ones(4)
    check(d, *call(op, d), reference(d))


def test_large_steps_stay_finite(op):
    """dt at the top of bf16: dt A overflows, dA is 0, and nothing of the state survives."""
    d = make([140], H=2, seed=8)
    d["dt"][[3, 70, 129]] = 3e4
    out, pool = call(op, d)
    assert torch.isfinite(out.double()).all() and torch.isfinite(pool.double()).all()
    check(d, out, pool, reference(d))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_neighbours_do_not_leak(op, bad):
    """Non-finite tokens of one prompt, of rows of no prompt and of a fresh prompt's old slot
    stay out of the other prompts."""
    d = make([100, 70, 129, 64], H=2, seed=9, lead=5, gap=9)
    d["fresh"] = torch.tensor([True, False, True, False])
    base = d["x"]._base
    base[:5] = bad
    base[-9:] = bad
    base[105:175] = bad  # prompt 1
    for k in ("dt",):
        d[k][:5] = bad
        d[k][-9:] = bad
    d["pool"][d["slots"][0]] = bad
    d["pool"][d["slots"][2]] = bad
    out, pool = call(op, d)
    keep = dict(d)
    y, state, Y, M = reference(keep, skip=(1,))
    rows = torch.cat([torch.arange(5, 105), torch.arange(175, 368)])
    assert torch.isfinite(out[rows].double()).all()
    s = d["slots"][[0, 2, 3]].long()
    err = (out.double() - y).abs()[rows]
    assert (err <= (2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -14) * Y + TINY)[rows]).all()
    assert ((pool.double() - state).abs()[s] <= M[s] * 2.0 ** -15).all()


@pytest.mark.parametrize("P", [64, 24])
def test_two_calls_continue_one(op, P):
    """A prompt cut anywhere gives the same state and readouts as in one call."""
    d = make([333], H=3, P=P, seed=10)
    d["fresh"] = torch.tensor([True])
    ref = reference(d)
    g = to_gpu(d)
    out = torch.full(g["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    for lo, hi, fresh in ((0, 1, 1), (1, 130, 0), (130, 130, 0), (130, 333, 0)):
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        ws = torch.empty(op.prompts_workspace_bytes(g["pool"], g["x"], g["B"], g["slots"]),
                         dtype=torch.uint8, device="cuda")
        op.prompts(g["pool"], g["slots"], cu, g["x"][lo:hi], g["dt"][lo:hi], g["dt_bias"],
                   g["A"], g["B"][lo:hi], g["C"][lo:hi], g["D"], out[lo:hi], ws,
                   fresh=torch.tensor([fresh], dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    check(d, out.cpu(), g["pool"].cpu(), ref)


def test_decode_step_continues_a_prompt(op):
    d = make([201], H=4, seed=11)
    ref = reference(d)
    g = to_gpu(d)
    out = torch.empty(g["x"].shape, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    ws = torch.empty(op.prompts_workspace_bytes(g["pool"], g["x"], g["B"], g["slots"]),
                     dtype=torch.uint8, device="cuda")
    op.prompts(g["pool"], g["slots"], cu, g["x"], g["dt"], g["dt_bias"], g["A"], g["B"], g["C"],
               g["D"], out, ws, fresh=g["fresh"])
    op(g["pool"], g["slots"], g["x"][200:], g["dt"][200:], g["dt_bias"], g["A"], g["B"][200:],
       g["C"][200:], g["D"], out[200:])
    torch.cuda.synchronize()
    check(d, out.cpu(), g["pool"].cpu(), ref)


def test_operands_without_alignment(op):
    """Rows that no 16-byte vector divides, element-strided tokens and expanded dt, A, D."""
    d = make([90, 41], H=2, P=40, N=128, seed=12)
    ref = reference(d)
    g = {k: v.cuda() for k, v in d.items()}
    T, H, P = d["x"].shape

    def odd(t, pad=1):
        big = torch.zeros(t.shape[0], t.shape[1], t.shape[2] + pad, dtype=t.dtype, device="cuda")
        big[..., pad:] = t
        return big[..., pad:]

    out = torch.full((T, H, P + 3), 7.0, dtype=torch.bfloat16, device="cuda")[..., 3:]
    dt = torch.zeros(T, 2 * H, dtype=torch.bfloat16, device="cuda")[:, ::2]
    dt.copy_(g["dt"])
    ws = torch.empty(op.prompts_workspace_bytes(g["pool"], g["x"], g["B"], g["slots"]),
                     dtype=torch.uint8, device="cuda")
    op.prompts(g["pool"], g["slots"], g["cu"], odd(g["x"]), dt[..., None].expand(T, H, P),
               g["dt_bias"][:, None].expand(H, P), g["A"][:, None, None].expand(H, P, 128),
               odd(g["B"]), odd(g["C"], 3), g["D"][:, None].expand(H, P), out, ws,
               fresh=g["fresh"])
    torch.cuda.synchronize()
    check(d, out.cpu(), g["pool"].cpu(), ref)


@pytest.mark.parametrize("P", [64, 8])
def test_strided_pool_and_slots(op, P):
    """The pool as a view with padding between rows, heads and slots; every other entry of the
    slot array."""
    d = make([130, 20], H=2, P=P, seed=13)
    ref = reference(d)
    g = to_gpu(d)
    n = d["pool"].shape[0]
    big = torch.full((n, 3, P + 2, 136), 3.0, device="cuda")
    pool = big[:, :2, :P, :128]
    pool.copy_(g["pool"])
    slots = torch.full((4,), -5, dtype=torch.int32, device="cuda")[::2]
    slots.copy_(g["slots"])
    out = torch.full(g["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(op.prompts_workspace_bytes(pool, g["x"], g["B"], slots), dtype=torch.uint8,
                     device="cuda")
    op.prompts(pool, slots, g["cu"], g["x"], g["dt"], g["dt_bias"], g["A"], g["B"], g["C"],
               g["D"], out, ws, fresh=g["fresh"])
    torch.cuda.synchronize()
    check(d, out.cpu(), pool.cpu(), ref)
    assert (big[:, 2] == 3.0).all() and (big[:, :, P:] == 3.0).all()
    assert (big[..., 128:] == 3.0).all()


@pytest.mark.parametrize("P", [64, 8])
def test_bad_prompts_are_skipped_and_counted(op, P):
    d = make([60, 130, 40, 7], H=2, P=P, seed=14)
    op.get_error()
    d["slots"][1] = d["pool"].shape[0]
    out, pool = call(op, d)
    check(d, out, pool, reference(d, skip=(1,)))
    assert op.get_error() == (1, 1)
    d["slots"][1] = -1
    d["cu"][4] = 10 ** 6  # the last prompt would end outside the call's rows
    out, pool = call(op, d)
    check(d, out, pool, reference(d, skip=(1, 3)))
    assert op.get_error() == (2, 1)


def test_offsets_that_run_backwards_are_skipped(op):
    d = make([60, 50, 40], H=2, seed=15)
    d["cu"] = torch.tensor([0, 60, 20, 150], dtype=torch.int32)
    # prompt 1 runs from 60 back to 20; prompt 2 from 20 overlaps prompt 0's rows: only count
    d["slots"][2] = -1
    op.get_error()
    out, pool = call(op, d)
    check(d, out, pool, reference(d, skip=(1, 2)))
    assert op.get_error() == (2, 1)


@pytest.mark.parametrize("P", [64, 8])
def test_no_tokens_at_all(op, P):
    """Only empty prompts: a fresh one's slot becomes zero, the other keeps its bits."""
    d = make([0, 0], H=2, P=P, seed=16)
    d["fresh"] = torch.tensor([True, False])
    out, pool = call(op, d)
    assert out.shape[0] == 0
    want = d["pool"].clone()
    want[d["slots"][0]] = 0
    assert torch.equal(pool, want)


def test_without_fresh_every_prompt_continues(op):
    d = make([40, 200], H=2, seed=17)
    out, pool = call(op, d, fresh=False)
    d["fresh"] = None
    check(d, out, pool, reference(d))


def test_same_call_same_bits(op):
    d = make([700, 130, 1], H=4, seed=18)
    a, b = call(op, d), call(op, d)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16))
    assert torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


def test_on_a_side_stream_and_in_a_graph(op):
    d = make([300, 64], H=2, seed=19)
    ref = reference(d)
    g = to_gpu(d)
    start = g["pool"].clone()
    out = torch.full(g["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(op.prompts_workspace_bytes(g["pool"], g["x"], g["B"], g["slots"]),
                     dtype=torch.uint8, device="cuda")
    args = (g["pool"], g["slots"], g["cu"], g["x"], g["dt"], g["dt_bias"], g["A"], g["B"],
            g["C"], g["D"], out, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op.prompts(*args, fresh=g["fresh"], stream=side)
    side.synchronize()
    check(d, out.cpu(), g["pool"].cpu(), ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.prompts(*args, fresh=g["fresh"])
    g["pool"].copy_(start)
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    check(d, out.cpu(), g["pool"].cpu(), ref)


@pytest.mark.parametrize("H,P,N,state,idx", [(8, 64, 128, torch.float32, torch.int32),
                                             (4, 128, 64, torch.bfloat16, torch.int64)])
def test_more_prompts_than_the_device_holds(op, H, P, N, state, idx):
    """Enough prompts (four pairs of columns each) that CTAs share the chunks of all of them and
    hand states on in the middle of a prompt; among them empty ones, one bad, one long."""
    lens = [500 + (97 * i) % 301 for i in range(39)]
    lens[5] = lens[6] = lens[38] = 0
    lens[7], lens[20], lens[21] = 1, 3100, 128
    d = make(lens, H=H, P=P, N=N, state=state, idx=idx, seed=29)
    d["fresh"][5], d["fresh"][6] = True, False
    d["slots"][11] = len(lens) + 50
    ref = reference(d, skip=(11,))
    out, pool = call(op, d)
    assert op.get_error() == (1, 11)
    check(d, out, pool, ref)
    again = call(op, d)
    assert op.get_error() == (1, 11)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16))
    assert torch.equal(pool.view(torch.int16), again[1].view(torch.int16))


@pytest.mark.parametrize("lens,N,H", [([300], 128, 2), ([70], 64, 4), ([128, 257], 128, 3),
                                      ([5003], 128, 2)], ids=str)
def test_no_token_reaches_back(op, lens, N, H):
    """An infinity or NaN in one element of x: what came before it, and every other row of the
    state, is as it would be without it; its own row is lost from that token on."""
    d = make(lens, H=H, N=N, seed=31)
    clean = call(op, d)
    lo, hi = d["cu"][-2].item(), d["cu"][-1].item()
    for k, (t, h, p) in enumerate([(lo + 3, 0, 5), (hi - 1, H - 1, 63), ((lo + hi) // 2, 1, 0)]):
        x = d["x"][t, h, p].clone()
        d["x"][t, h, p] = (float("nan"), float("inf"), -float("inf"))[k]
        out, pool = call(op, d)
        keep = torch.ones_like(out, dtype=torch.bool)
        keep[t:hi, h, p] = False
        assert torch.equal(out[keep], clean[0][keep]) and not out[~keep].isfinite().any()
        state = torch.ones_like(pool, dtype=torch.bool)
        state[d["slots"][-1].item(), h, p] = False
        assert torch.equal(pool[state], clean[1][state]) and not pool[~state].isfinite().any()
        d["x"][t, h, p] = x


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("slow", [False, True])
def test_an_fp32_state_is_carried_in_fp32(op, N, slow):
    """Relative 2-norm of a head's state within 2^-21.1 of the recurrence in fp64: some ten
    roundings per term (dt, its exponent and power, the products, the sums), each 2^-24 / sqrt(3)
    in the mean square and independent, come to 2^-23.1; four times that.  A token's weight cut
    to two bf16 parts alone is 2^-20 off.  Lengths end in every part of a chunk."""
    d = make([1, 17, 37, 64, 65, 100, 128, 150, 300], H=4, N=N, seed=23)
    if slow:
        d["A"] = d["A"] * 2.0 ** -7
    pool = call(op, d)[1].double()
    _, want, _, _ = reference(d)
    off = ((pool - want).square().sum((2, 3)) / want.square().sum((2, 3))).sqrt()[d["slots"]]
    assert off.max() <= 2.0 ** -21.1, off.amax(1)


def test_refusals(op):
    d = to_gpu(make([40], H=2, seed=20))
    out = torch.empty(d["x"].shape, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(op.prompts_workspace_bytes(d["pool"], d["x"], d["B"], d["slots"]),
                     dtype=torch.uint8, device="cuda")

    def attempt(error, **change):
        a = dict(d, out=out, ws=ws)
        a.update(change)
        with pytest.raises(error):
            op.prompts(a["pool"], a["slots"], a["cu"], a["x"], a["dt"], a["dt_bias"], a["A"],
                       a["B"], a["C"], a["D"], a["out"], a["ws"], fresh=a["fresh"])

    attempt(TypeError, x=d["x"].float())
    attempt(TypeError, cu=d["cu"].long())
    attempt(TypeError, slots=d["slots"].float())
    attempt(ValueError, cu=d["cu"][:1])
    attempt(ValueError, out=out[:-1])
    attempt(ValueError, B=d["B"][:, :, :64])
    attempt(ValueError, dt=d["dt"][:-1])
    attempt(ValueError, x=d["x"].cpu())
    attempt(ValueError, fresh=d["fresh"].cpu())
    attempt(ValueError, fresh=d["fresh"].repeat(2))
    attempt(ssu.SsuError, dt=d["dt"][:, :, None].repeat(1, 1, 64))  # not constant over headdim
    attempt(ssu.SsuError, x=d["x"].transpose(1, 2).contiguous().transpose(1, 2))
    attempt(ssu.SsuError, pool=d["pool"][..., :32].contiguous(), B=d["B"][..., :32].contiguous(),
            C=d["C"][..., :32].contiguous())
    if ws.numel():
        attempt(ssu.SsuError, ws=ws[:-256])
        attempt(ssu.SsuError, ws=None)
    torch.cuda.synchronize()
    assert op.get_error() == (0, -1)
