"""The gated delta rule (``ssu_delta_update``, ``ssu_delta_prompts``) against the recurrence in
fp64, token by token.

Tolerances, derived before any run.  An error of a state's row p passes on through a (1 - beta kn
kn^T), which makes no vector longer (0 <= beta <= 1, |kn| <= 1), so errors add up at most, each
forgotten with the decay.  With R_p the largest |S_p| + |v_p| (2-norm of the row) that a prompt
meets, one token adds at most 2^-20 R_p: products of 128 terms in a tree (2^-20.5 |S_p| by
Cauchy-Schwarz), lengths, decay and gate from exp and softplus (2^-22 each), two roundings of the
update.  The chunked form keeps its parts of operands to 2^-17 of products that reach the state
through at most one chunk, and stays below that sum.  With a_max the largest decay of the inputs,
n = min(tokens, 1 / (1 - a_max)) tokens' errors are alive at a time:

* fp32 state: row errors up to n 2^-20 R_p, and over a whole call of random signs 2^-17 of the
  2-norm of the states that the call wrote.
* bf16 state: 2^-8 |S| more (its own rounding; half a step).
* readout: with M the magnitudes (M <- a M + |e kn|) and Y = M |qn|, 2^-8 |y| (its own rounding)
  and, where the chunked form rounds a chunk's weights and corrections to bf16 once each,
  (2 * 2^-8 + 2^-13) Y; over a whole call of random signs the roundings add as squares, so the
  relative 2-norm stays within 2^-8.
"""

from __future__ import annotations

import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import selective_state_update_02_gb300 as ssu  # noqa: E402
from test_guards_gpu import Guarded  # noqa: E402

EPS = 1e-6


@pytest.fixture(scope="module")
def op():
    handle = ssu.SelectiveStateUpdate(0)
    yield handle
    torch.cuda.synchronize()
    handle.close()


def make(lens, H=4, P=128, N=128, G=2, state=torch.float32, seed=0, idx=torch.int32, extra=3,
         lead=0, gap=0, keys="silu"):
    """Inputs of a call on the GPU; ``lead`` rows before the first prompt and ``gap`` rows after
    the last are no prompt's.  For a decode step every prompt has one token."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    bs, T = len(lens), lead + sum(lens) + gap
    qkv = normal(T, 2 * G * N + H * P)
    if keys == "silu":  # a common part in all keys
        qkv = torch.nn.functional.silu(qkv)
    elif keys == "same":  # every key of a head the same: the hardest triangular systems
        qkv[:, G * N:2 * G * N] = qkv[:1, G * N:2 * G * N].clone()
    qkv = qkv.bfloat16()
    return dict(
        pool=(0.1 * normal(bs + extra, H, P, N)).to(state),
        slots=torch.randperm(bs + extra, generator=g, device="cuda")[:bs].to(idx),
        cu=torch.tensor([lead] + [lead + s for s in itertools.accumulate(lens)]).to(idx).cuda(),
        q=qkv[:, :G * N].view(T, G, N), k=qkv[:, G * N:2 * G * N].view(T, G, N),
        v=qkv[:, 2 * G * N:].view(T, H, P),
        dt=(torch.rand(T, H, generator=g, device="cuda") * 4 - 4).bfloat16(),
        dt_bias=torch.rand(H, generator=g, device="cuda") * 2 - 1,
        A=-torch.exp(torch.rand(H, generator=g, device="cuda") * 2.77),
        b=normal(T, H).bfloat16(), fresh=torch.rand(bs, generator=g, device="cuda") < 0.5)


def reference(d, skip=(), scale=None, eps=EPS):
    """The recurrence in fp64: readouts and states, the magnitudes Y and R of the tolerances, and
    the largest decay; what a call must not touch keeps its start values (readouts: NaN)."""
    H, N = d["v"].shape[1], d["q"].shape[2]
    of = torch.arange(H, device="cuda") // (H // d["q"].shape[1])
    scale = N ** -0.5 if scale is None else scale

    def unit(t):
        t = t.double()
        if eps is not None:
            t = t / torch.sqrt((t * t).sum(-1, keepdim=True) + eps)
        return t[:, of]

    q, k, v = scale * unit(d["q"]), unit(d["k"]), d["v"].double()
    z = d["dt"].double() + d["dt_bias"].double()
    a = torch.exp(torch.nn.functional.softplus(z, threshold=700.0) * d["A"].double())
    beta = torch.sigmoid(d["b"].double())
    pool = d["pool"].double()
    y, Y = torch.full_like(v, float("nan")), torch.zeros_like(v)
    R = torch.zeros(pool.shape[:3], dtype=torch.float64, device="cuda")
    cu = d["cu"].tolist()
    most = 0.0
    for i, slot in enumerate(d["slots"].tolist()):
        if i in skip:
            continue
        S = pool[slot].clone()
        if d["fresh"] is not None and d["fresh"][i]:
            S.zero_()
        M, worst = S.abs(), S.norm(dim=-1)
        for t in range(cu[i], cu[i + 1]):
            at = a[t][:, None, None]
            e = beta[t][:, None] * (v[t] - a[t][:, None] * (S @ k[t][..., None])[..., 0])
            step = e[..., None] * k[t][:, None]
            S = S * at + step
            M = M * at + step.abs()
            y[t] = (S @ q[t][..., None])[..., 0]
            Y[t] = (M @ q[t].abs()[..., None])[..., 0]
            worst = torch.maximum(worst, S.norm(dim=-1) + v[t].abs())
        if cu[i] < cu[i + 1]:
            most = max(most, a[cu[i]:cu[i + 1]].max().item())
        pool[slot], R[slot] = S, worst
    return y, pool, Y, R, most


def call(op, d, fresh=True, out=None, **kw):
    """Readouts and the pool of a prompt call, on copies."""
    pool = d["pool"].clone()
    out = torch.full(d["v"].shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = torch.full((op.delta_workspace_bytes(pool, d["v"], d["k"], d["slots"]),), 0xff,
                    dtype=torch.uint8, device="cuda")
    op.delta_prompts(pool, d["slots"], d["cu"], d["q"], d["k"], d["v"], d["dt"], d["dt_bias"],
                     d["A"], d["b"], out, ws, fresh=d["fresh"] if fresh else None, **kw)
    torch.cuda.synchronize()
    return out, pool


def check(d, out, pool, ref, chunked=True):
    y, want, Y, R, most = ref
    run = ~torch.isnan(y)
    assert (out[~run] == 7.0).all(), "rows of no prompt were written"
    err = (out.double() - y).abs()[run]
    tol = (2.0 ** -8 * y.abs() + (2.0 ** -7 * chunked + 2.0 ** -13) * Y + 2.0 ** -126)[run]
    assert (err <= tol).all(), f"readout off by {(err / tol).max():.3g} of its tolerance"
    if run.sum() >= 4096:
        rel = err.norm() / y[run].norm()
        assert rel <= 2.0 ** -8, f"readout 2-norm {rel:.3g}"
    err = (pool.double() - want).abs()
    touched = torch.zeros(len(pool), dtype=torch.bool, device="cuda")
    touched[d["slots"].long()] = True
    assert torch.equal(pool[~touched], d["pool"][~touched])
    if pool.dtype == torch.bfloat16:
        err = (err - 2.0 ** -8 * want.abs()).clamp_min(0.0)
    elif want[touched].numel() >= 4096:
        rel = err[touched].norm() / want[touched].norm().clamp_min(1e-30)
        assert rel <= 2.0 ** -17, f"state 2-norm {rel:.3g}"
    n = min(max(1, len(d["v"])), 1.0 / max(1e-9, 1.0 - most))
    tol = n * 2.0 ** -20 * R + 2.0 ** -126
    rows = err.norm(dim=-1)
    assert (rows <= tol).all(), f"state row off by {(rows / tol).max():.3g} of its tolerance"


LENS = [
    [1], [2], [16], [31], [37], [63], [64], [65], [127], [128], [129], [300], [1000],
    [1, 0, 5, 64, 129, 0, 77], [256, 3, 400], [16] * 40,
]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [64, 128])
def test_lengths(op, lens, N, state):
    d = make(lens, N=N, state=state, seed=len(lens) + sum(lens))
    check(d, *call(op, d), reference(d))


@pytest.mark.parametrize("H,P,N,G", [
    (8, 64, 128, 8), (6, 64, 128, 2), (4, 256, 128, 1), (3, 64, 256, 1), (2, 80, 128, 1),
    (5, 3, 64, 1), (2, 192, 64, 2), (1, 1, 128, 1), (4, 64, 64, 4), (2, 72, 256, 2),
    (16, 128, 128, 8), (8, 128, 64, 1), (2, 320, 128, 2)], ids=str)
@pytest.mark.parametrize("idx", [torch.int32, torch.int64], ids=["i32", "i64"])
def test_shapes(op, H, P, N, G, idx):
    d = make([150, 0, 33], H, P, N, G, seed=H * P + N, idx=idx)
    check(d, *call(op, d), reference(d))


@pytest.mark.parametrize("keys", ["normal", "same"])
def test_keys(op, keys):
    """Keys in every direction, and all of a head's keys the same with gates near one."""
    d = make([200, 65], seed=3, keys=keys)
    if keys == "same":
        d["b"] = torch.full_like(d["b"], 6.0)
    check(d, *call(op, d), reference(d))


@pytest.mark.parametrize("kind", ["strong", "none", "weak", "mixed"])
@pytest.mark.parametrize("N", [64, 128])
def test_decays(op, kind, N):
    """a that underflows to 0, a that is exactly 1, slow decays, and both within a chunk."""
    d = make([400, 129], N=N, seed=7)
    g = torch.Generator(device="cuda").manual_seed(1)
    if kind == "strong":
        d["dt"] = torch.where(torch.rand(d["dt"].shape, generator=g, device="cuda") < 0.3, 60.0,
                              2.0).bfloat16()
        d["A"] = torch.tensor([-16.0, -8.0, -2.0, -0.5], device="cuda")
    elif kind == "none":
        d["dt"] = torch.full_like(d["dt"], -200.0)
    elif kind == "weak":
        d["dt"] = torch.full_like(d["dt"], -4.0)
        d["A"] = -torch.ones(4, device="cuda")
    else:
        d["dt"] = torch.where(torch.rand(d["dt"].shape, generator=g, device="cuda") < 0.1, 100.0,
                              -6.0).bfloat16()
        d["A"] = torch.tensor([-16.0, -4.0, -1.0, -0.25], device="cuda")
    check(d, *call(op, d), reference(d))


@pytest.mark.parametrize("gate", [-200.0, 200.0])
def test_gates(op, gate):
    """beta of exactly 0 (the state only decays) and 1 (the key's value is replaced)."""
    d = make([130, 70], seed=11)
    d["b"] = torch.full_like(d["b"], gate)
    check(d, *call(op, d), reference(d))


@pytest.mark.parametrize("scale,eps", [(1.0, EPS), (0.3, 0.0), (0.05, None)])
def test_scale_and_lengths(op, scale, eps):
    """Other scales; keys and queries left as they are (short enough that the rule is stable)."""
    d = make([100, 65], seed=13)
    if eps is None:
        d["k"] = (d["k"] / (d["k"].float().norm(dim=-1, keepdim=True) * 1.1)).bfloat16()
    check(d, *call(op, d, scale=scale, qk_eps=eps), reference(d, scale=scale, eps=eps))


def test_a_call_in_parts_continues(op):
    """A prompt cut into calls of odd lengths ends where the whole one does."""
    d = make([333], seed=17)
    d["fresh"] = None
    ref = reference(d)
    pool = d["pool"].clone()
    outs = []
    for lo, hi in ((0, 5), (5, 70), (70, 199), (199, 333)):
        part = {k: d[k][lo:hi] for k in ("q", "k", "v", "dt", "b")}
        part.update(pool=pool, slots=d["slots"], dt_bias=d["dt_bias"], A=d["A"], fresh=None,
                    cu=torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"))
        out, pool = call(op, part, fresh=False)
        outs.append(out)
    check(d, torch.cat(outs), pool, ref)


def step(op, d, pool, out, at=None, **kw):
    at = slice(None) if at is None else at
    op.delta(pool, d["slots"], d["q"][at], d["k"][at], d["v"][at], d["dt"][at], d["dt_bias"],
             d["A"], d["b"][at], out, **kw)


@pytest.mark.parametrize("bs,H,P,N,G", [
    (1, 4, 128, 128, 2), (7, 4, 128, 128, 4), (61, 8, 64, 64, 2), (5, 3, 40, 256, 1),
    (3, 2, 1, 64, 1), (2, 5, 130, 128, 5), (300, 2, 64, 128, 1)], ids=str)
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("idx", [torch.int32, torch.int64], ids=["i32", "i64"])
def test_one_token(op, bs, H, P, N, G, state, idx):
    d = make([1] * bs, H, P, N, G, state=state, seed=bs + P, idx=idx)
    d["fresh"] = None
    pool, out = d["pool"].clone(), torch.full(d["v"].shape, 7.0, dtype=torch.bfloat16,
                                              device="cuda")
    step(op, d, pool, out)
    torch.cuda.synchronize()
    check(d, out, pool, reference(d), chunked=False)


def test_tokens_continue_prompts(op):
    """A prompt, then its last tokens one by one: the readouts and states of the whole one."""
    d = make([140, 70, 3], seed=19)
    d["fresh"] = torch.ones(3, dtype=torch.bool, device="cuda")
    y, want, Y, R, most = reference(d)
    cu = d["cu"].tolist()
    short = dict(d)
    keep = [i for b in range(3) for i in range(cu[b], cu[b + 1] - 2)]
    for k in ("q", "k", "v", "dt", "b"):
        short[k] = d[k][keep]
    short["cu"] = torch.tensor([0, 138, 206, 207], dtype=torch.int32, device="cuda")
    _, pool = call(op, short)
    got = torch.full_like(d["v"], 7.0)
    for b in range(3):
        got[cu[b]:cu[b + 1] - 2] = 0
    for n in (2, 1):
        rows = d["cu"][1:].long() - n
        out = torch.empty_like(d["v"][rows])
        step(op, d, pool, out, rows)
        got[rows] = out
    rows = torch.cat([d["cu"][1:].long() - 2, d["cu"][1:].long() - 1])
    err = (got.double() - y)[rows].abs()
    assert (err <= 2.0 ** -8 * y[rows].abs() + 2.0 ** -13 * Y[rows]).all()
    n = min(140, 1.0 / (1.0 - most))
    assert ((pool.double() - want).norm(dim=-1) <= n * 2.0 ** -20 * R).all()


def test_strided_operands(op):
    """Views with gaps everywhere: a wider activation, every second slot, head and row of a pool,
    an out inside a larger array."""
    H, P, N, G, lens = 4, 128, 128, 2, [70, 5, 200]
    d = make(lens, H, P, N, G, seed=23)
    T = sum(lens)
    wide = torch.zeros(T, 2 * G * (N + 8) + H * (P + 16), dtype=torch.bfloat16, device="cuda")
    e = dict(d)
    at = 0
    for k, heads, size, pad in (("q", G, N, 8), ("k", G, N, 8), ("v", H, P, 16)):
        view = wide[:, at:at + heads * (size + pad)].view(T, heads, size + pad)[..., :size]
        view.copy_(d[k])
        e[k], at = view, at + heads * (size + pad)
    dt, b = torch.zeros(2, H, T + 3, dtype=torch.bfloat16, device="cuda")
    dt[:, :T], b[:, :T] = d["dt"].t(), d["b"].t()
    e["dt"], e["b"] = dt[:, :T].t(), b[:, :T].t()
    room = torch.full((2 * len(d["pool"]), 2 * H, 2 * P, N), 3.0, device="cuda")
    room[::2, ::2, ::2] = d["pool"]
    e["slots"] = torch.stack([d["slots"], d["slots"]], 1)[:, 0]
    out = torch.full((T, 2 * H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(op.delta_workspace_bytes(room[::2, ::2, ::2], e["v"], e["k"], e["slots"]),
                     dtype=torch.uint8, device="cuda")
    op.delta_prompts(room[::2, ::2, ::2], e["slots"], d["cu"], e["q"], e["k"], e["v"], e["dt"],
                     d["dt_bias"], d["A"], e["b"], out[:, 1::2], ws, fresh=d["fresh"])
    torch.cuda.synchronize()
    assert (out[:, ::2] == 7.0).all() and (room[1::2] == 3.0).all()
    assert (room[:, 1::2] == 3.0).all() and (room[:, :, 1::2] == 3.0).all()
    check(d, out[:, 1::2].contiguous(), room[::2, ::2, ::2].contiguous(), reference(d))


@pytest.mark.parametrize("shift", [1, 3])
def test_unaligned_operands(op, shift):
    """q, k, v and out at odd addresses, head strides that are no multiple of 16 bytes."""
    d = make([100, 37], seed=29)
    for k in ("q", "k", "v"):
        t = d[k]
        flat = torch.zeros(t.numel() + shift + t.shape[0], dtype=t.dtype, device="cuda")
        view = flat[shift:].as_strided(t.shape, (t.shape[1] * t.shape[2] + 1, t.shape[2], 1))
        view.copy_(t)
        d[k] = view
    check(d, *call(op, d), reference(d))


def test_bad_prompts_and_slots_are_skipped(op):
    d = make([70, 30, 40, 65], seed=31, lead=4, gap=6)
    d["slots"][1] = len(d["pool"])
    d["slots"][2] = -1
    op.get_error()
    out, pool = call(op, d)
    assert op.get_error() == (2, 1)
    ref = reference(d, skip=(1, 2))
    d["slots"] = d["slots"][[0, 3]]
    check(d, out, pool, ref)


@pytest.mark.parametrize("cu", [[150, 0, 64, 128], [0, 500, 64, 90], [-3, 20, 64, 128],
                                [90, 40, 40, 130], [200, 199, 3, 201]], ids=str)
def test_offsets_out_of_order(op, cu):
    """Bad prompts are left out; the others are right."""
    d = make([100, 50, 50], seed=37)
    d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    skip = [b for b in range(3) if not 0 <= cu[b] <= cu[b + 1] <= 200]
    op.get_error()
    out, pool = call(op, d)
    assert op.get_error() == (len(skip), skip[0])
    keep = [b for b in range(3) if b not in skip]
    ref = reference(d, skip=skip)
    d["slots"] = d["slots"][keep]
    check(d, out, pool, ref)


@pytest.mark.parametrize("where", ["q", "k", "v", "dt", "b"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nothing_before_a_bad_token_changes(op, where, bad):
    """An infinity or NaN in one token's operand: the readouts before it, other prompts' and, for a
    value, other rows' are as without it, and rows of no prompt reach nothing."""
    d = make([100, 70, 129], seed=41, lead=5, gap=9)
    clean_out, clean_pool = call(op, d)
    e = {k: (v.clone() if k in ("q", "k", "v", "dt", "b", "pool") else v) for k, v in d.items()}
    for row in (0, 4, len(d["v"]) - 1):  # rows of no prompt
        e[where][row] = bad
    t = d["cu"][2].item() + 80  # token 80 of the last prompt
    if where == "v":
        e["v"][t, 1, 7] = bad
    else:
        e[where][t, 0] = bad
    out, pool = call(op, e)
    last = d["slots"][2].item()
    others = [i for i in range(len(pool)) if i != last]
    assert torch.equal(pool[others], clean_pool[others])

    def near(a, b):  # the chunk with the token may take another form: same to rounding
        return ((a.double() - b.double()).abs() <=
                2.0 ** -6 * b.double().abs() + 2.0 ** -6 * b.double().abs().max()).all()

    assert near(out[:t], clean_out[:t])
    assert torch.equal(out[d["cu"][0]:d["cu"][2]], clean_out[d["cu"][0]:d["cu"][2]])
    if where == "v":
        keep = torch.ones(out.shape[1:], dtype=torch.bool, device="cuda")
        keep[1, 7] = False
        assert near(out[t:][:, keep], clean_out[t:][:, keep])
        assert not torch.isfinite(out[t:len(out) - 9, 1, 7]).any()
        assert torch.isfinite(pool[last][keep]).all()
        assert not torch.isfinite(pool[last, 1, 7]).all()
    elif where == "q":
        heads = range(0, 2)  # of key head 0
        assert all(not torch.isfinite(out[t, h]).any() for h in heads) or bad == float("inf")
        assert near(out[t + 1:], clean_out[t + 1:]) and torch.isfinite(pool).all()
    elif not (bad == float("inf") and where in ("b", "dt")):  # (those have finite limits)
        assert not torch.isfinite(out[t, 0]).any() and not torch.isfinite(pool[last, 0]).all()
    else:
        check_inf = torch.isfinite(out[t:len(out) - 9])
        assert check_inf.all()


def test_bad_states_stay_in_their_rows(op):
    """An infinity or NaN in a slot's state reaches its own row's readouts alone; a fresh prompt does
    not read its slot, and a slot of no prompt reaches nothing."""
    d = make([100, 70], seed=43)
    d["fresh"] = torch.tensor([False, True], device="cuda")
    clean_out, clean_pool = call(op, d)
    e = dict(d, pool=d["pool"].clone())
    s0, s1 = d["slots"].tolist()
    free = next(i for i in range(len(d["pool"])) if i not in (s0, s1))
    e["pool"][s0, 2, 5, 9] = float("nan")
    e["pool"][s1] = float("nan")
    e["pool"][free] = float("inf")
    out, pool = call(op, e)
    keep = torch.ones(out.shape[1:], dtype=torch.bool, device="cuda")
    keep[2, 5] = False
    assert torch.equal(out[100:], clean_out[100:]) and torch.equal(pool[s1], clean_pool[s1])
    assert torch.equal(out[:100][:, keep], clean_out[:100][:, keep])
    assert not torch.isfinite(out[:100, 2, 5]).any()
    assert torch.equal(pool[s0][keep], clean_pool[s0][keep])


def test_empty_calls(op):
    d = make([], seed=47)
    out, pool = call(op, d)
    assert torch.equal(pool, d["pool"])
    d = make([0, 0], seed=48)
    d["fresh"] = torch.tensor([True, False], device="cuda")
    out, pool = call(op, d)
    assert (pool[d["slots"][0].long()] == 0).all()
    rest = [i for i in range(len(pool)) if i != d["slots"][0].item()]
    assert torch.equal(pool[rest], d["pool"][rest])
    step(op, make([]), make([])["pool"], torch.empty(0, 4, 128, dtype=torch.bfloat16,
                                                     device="cuda"))


def test_replayed_graphs_and_other_streams(op):
    """A captured prompt call and decode step, replayed on changed inputs on another stream, give
    the bits of plain calls; two handles with a workspace each run side by side."""
    d = make([200, 65, 3], seed=53)
    ws = torch.empty(op.delta_workspace_bytes(d["pool"], d["v"], d["k"], d["slots"]),
                     dtype=torch.uint8, device="cuda")
    pool, out = d["pool"].clone(), torch.zeros_like(d["v"])
    rows = d["cu"][1:].long() - 1
    one = {k: d[k][rows].clone() for k in ("q", "k", "v", "dt", "b")}
    one_out = torch.zeros_like(one["v"])

    def both(o=op):
        o.delta_prompts(pool, d["slots"], d["cu"], d["q"], d["k"], d["v"], d["dt"], d["dt_bias"],
                        d["A"], d["b"], out, ws, fresh=d["fresh"])
        o.delta(pool, d["slots"], one["q"], one["k"], one["v"], one["dt"], d["dt_bias"], d["A"],
                one["b"], one_out)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for n in range(3):
        start = make([200, 65, 3], seed=60 + n)
        for k in ("q", "k", "v", "dt", "b"):
            d[k].copy_(start[k])
        pool.copy_(start["pool"])
        both()
        torch.cuda.synchronize()
        want = [t.clone() for t in (pool, out, one_out)]
        pool.copy_(start["pool"])
        out.zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (pool, out, one_out)))


def test_the_same_bits_again_and_without_dependent_launch(op):
    d = make([300, 64, 1, 90], seed=71)
    a = call(op, d)
    b = call(op, d)
    ssu.ssu_set_pdl(op.handle, False)
    try:
        c = call(op, d)
    finally:
        ssu.ssu_set_pdl(op.handle, True)
    for other in (b, c):
        assert all(torch.equal(x, y) for x, y in zip(a, other))


@pytest.mark.parametrize("cu,skip", [([0, 80, 60, 200], [1, 2]), ([0, 200, 100, 150], [1, 2]),
                                     ([0, 64, 0, 200], [1, 2]), ([10, 10, 5, 5], [1])], ids=str)
def test_prompts_that_overlap(op, cu, skip):
    """Where offsets run backwards, a chunked prompt that begins before the end of a good one
    before it is left out like a bad one."""
    d = make([100, 50, 50], seed=39)
    d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    op.get_error()
    out, pool = call(op, d)
    assert op.get_error() == (len(skip), skip[0])
    ref = reference(d, skip=skip)
    d["slots"] = d["slots"][[b for b in range(3) if b not in skip]]
    check(d, out, pool, ref)


@pytest.mark.parametrize("A", [0.02, 0.7])
def test_growing_states(op, A):
    """Decays above one: within a chunk's range, and past it (such chunks go token by token)."""
    d = make([150, 70], seed=73)
    d["A"] = torch.full_like(d["A"], A)
    d["dt"] = torch.full_like(d["dt"], 0.5)
    out, pool = call(op, d)
    y, want, Y, R, most = reference(d)
    # With 0.7 a state grows by up to 3.18 a token: 150 of them are a factor of 2^250, which fp32 does
    # not hold.  Heads are compared up to where their magnitudes pass 2^100, and their states where
    # they never do.
    cu = d["cu"].tolist()
    for i, slot in enumerate(d["slots"].tolist()):
        rows = slice(cu[i], cu[i + 1])
        size = Y[rows].amax(-1).cummax(0).values  # [tokens, H]
        keep = size < 2.0 ** 100
        err = (out[rows].double() - y[rows]).abs()
        tol = 2.0 ** -8 * y[rows].abs() + (2.0 ** -7 + 2.0 ** -13) * Y[rows]
        assert (err <= tol)[keep].all()
        whole = keep.all(0) & (R[slot].amax(-1) < 2.0 ** 100)
        rows_off = (pool[slot].double() - want[slot]).norm(dim=-1)
        assert (rows_off <= (cu[i + 1] - cu[i]) * 2.0 ** -20 * R[slot])[whole].all()
        assert A > 0.1 or whole.all()


def test_many_prompts(op):
    """More prompts than a warp has lanes and than a sort takes, bad ones and empty ones among
    them: nothing of one in another."""
    lens = [(37 * i) % 131 if i % 9 else 0 for i in range(70)]
    d = make(lens, H=2, G=1, seed=79)
    d["slots"][5] = -1
    check_some(op, d, skip=(5,))
    lens = [1 + (i * i) % 7 for i in range(1100)]
    d = make(lens, H=1, P=64, N=64, G=1, seed=83)
    check_some(op, d)


def check_some(op, d, skip=()):
    op.get_error()
    out, pool = call(op, d)
    assert op.get_error() == (len(skip), min(skip, default=-1))
    ref = reference(d, skip=skip)
    keep = [b for b in range(len(d["slots"])) if b not in skip]
    d["slots"] = d["slots"][keep]
    check(d, out, pool, ref)


def test_slots_past_32_bits(op):
    """A pool of more than 2^31 elements: its last slot, by prompts in both forms and one token."""
    H, P, N = 32, 128, 128
    slots = 2 ** 31 // (H * P * N) + 3
    pool = torch.zeros(slots, H, P, N, device="cuda")
    for tokens in (200, 20):
        d = make([tokens], H, P, N, G=16, seed=tokens, extra=0)
        d["fresh"] = None
        pool[-1] = d["pool"][0]
        y, want, Y, R, most = reference(d)
        out = torch.zeros_like(d["v"])
        at = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
        ws = torch.empty(op.delta_workspace_bytes(pool, d["v"], d["k"], at), dtype=torch.uint8,
                         device="cuda")
        op.delta_prompts(pool, at, d["cu"], d["q"], d["k"], d["v"], d["dt"], d["dt_bias"], d["A"],
                         d["b"], out, ws)
        check(d, out, pool[-1:].clone(), (y, want, Y, R, most))
        assert (pool[:-1] == 0).all()
    d = make([1], H, P, N, G=16, seed=89, extra=0)
    d["fresh"] = None
    pool[-1] = d["pool"][0]
    out = torch.zeros_like(d["v"])
    step(op, dict(d, slots=at), pool, out)
    check(d, out, pool[-1:].clone(), reference(d), chunked=False)
    assert (pool[:-1] == 0).all()


def test_batches_past_the_grid(op):
    """More requests than a grid's third dimension has."""
    bs = 66000
    d = make([1] * bs, H=1, P=8, N=64, G=1, seed=97, extra=0)
    pool, out = d["pool"].clone(), torch.zeros_like(d["v"])
    step(op, d, pool, out)
    pick = [0, 1, 65534, 65535, 65536, bs - 1]
    part = {k: d[k][pick] for k in ("q", "k", "v", "dt", "b")}
    part.update(slots=torch.arange(6, dtype=torch.int32, device="cuda"), dt_bias=d["dt_bias"],
                A=d["A"], pool=d["pool"][d["slots"][pick].long()], fresh=None,
                cu=torch.arange(7, dtype=torch.int32, device="cuda"))
    check(part, out[pick], pool[d["slots"][pick].long()], reference(part), chunked=False)


KINDS = {"few": dict(lens=[1, 0, 129, 64], H=4), "many": dict(lens=[65 + i for i in range(40)], H=2),
         "bf16": dict(lens=[300, 130], H=4, P=72, N=64, state=torch.bfloat16),
         "by token": dict(lens=[20, 150], H=3, P=24, N=256, G=3)}


@pytest.mark.parametrize("kind", KINDS)
def test_calls_stay_in_their_buffers(op, kind):
    """Canaries on both sides of the pool, the readouts and the workspace."""
    d = make(seed=101, extra=0, **KINDS[kind])
    d["slots"][0] = len(d["pool"])  # one prompt is skipped
    out, pool = call(op, d)
    n = op.delta_workspace_bytes(d["pool"], d["v"], d["k"], d["slots"])
    guards = [Guarded(t) for t in (d["pool"], torch.full_like(out, 7.0),
                                   torch.zeros(n, dtype=torch.uint8, device="cuda"))]
    room, y, ws = (g.t for g in guards)
    op.delta_prompts(room, d["slots"], d["cu"], d["q"], d["k"], d["v"], d["dt"], d["dt_bias"],
                     d["A"], d["b"], y, ws, fresh=d["fresh"])
    assert op.get_error() == (2, 0)
    assert all(g.intact() for g in guards)
    assert torch.equal(room, pool) and torch.equal(y, out)
    rows = d["cu"][1:].long() - 1
    one = torch.zeros_like(d["v"][rows])
    guard = Guarded(one)
    step(op, d, room, guard.t, rows)
    assert op.get_error() == (1, 0) and guard.intact() and guards[0].intact()


def test_calls_side_by_side(op):
    """Two handles on two streams with a workspace each; and two captured graphs that share one,
    replayed one after the other: the bits of calls alone."""
    ds = [make([150, 65, 200], seed=103), make([90, 300], seed=107)]
    want = [call(op, d) for d in ds]
    other = ssu.SelectiveStateUpdate(0)
    for _ in range(3):
        got = []
        for d, o in zip(ds, (op, other)):
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                pool, out = d["pool"].clone(), torch.full_like(d["v"], 7.0)
                ws = torch.empty(o.delta_workspace_bytes(pool, d["v"], d["k"], d["slots"]),
                                 dtype=torch.uint8, device="cuda")
                o.delta_prompts(pool, d["slots"], d["cu"], d["q"], d["k"], d["v"], d["dt"],
                                d["dt_bias"], d["A"], d["b"], out, ws, fresh=d["fresh"])
                got.append((out, pool, ws))
        torch.cuda.synchronize()
        for (out, pool, _), (y, state) in zip(got, want):
            assert torch.equal(out, y) and torch.equal(pool, state)
    n = max(op.delta_workspace_bytes(d["pool"], d["v"], d["k"], d["slots"]) for d in ds)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, results = [], []
    for d in ds:
        pool, out = d["pool"].clone(), torch.full_like(d["v"], 7.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op.delta_prompts(pool, d["slots"], d["cu"], d["q"], d["k"], d["v"], d["dt"],
                             d["dt_bias"], d["A"], d["b"], out, ws, fresh=d["fresh"])
        graphs.append(graph)
        results.append((out, pool))
    for _ in range(2):
        for d, graph, (out, pool), (y, state) in zip(ds, graphs, results, want):
            pool.copy_(d["pool"])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, y) and torch.equal(pool, state)
    assert op.get_error() == (0, -1) and other.get_error() == (0, -1)
    other.close()


@pytest.mark.parametrize("P,N,state", [(72, 64, torch.bfloat16), (192, 128, torch.float32)], ids=str)
@pytest.mark.parametrize("where", ["k", "v", "dt"])
def test_bad_tokens_of_other_sizes(op, P, N, state, where):
    """Chunks taken token by token where a CTA's rows are not all the head's, and in two slabs."""
    d = make([100, 150], P=P, N=N, state=state, seed=109)
    y, want, Y, R, most = reference(d)
    t = 170  # token 70 of the second prompt: the rows before it are as the formula gives them
    d[where][(t, 0, 3) if where == "v" else (t, 0)] = float("nan")
    out, pool = call(op, d)
    tol = 2.0 ** -8 * y.abs() + (2.0 ** -7 + 2.0 ** -13) * Y
    assert ((out.double() - y).abs() <= tol)[:t].all()
    assert torch.isnan(out[t:, 0, 3]).all()
    other = torch.ones(4, dtype=torch.bool, device="cuda")
    other[:2] = False  # the heads of key head 0; for a value and a decay more is right, below
    assert ((out.double() - y).abs() <= tol)[t:][:, other].all()
    if where != "k":
        assert ((out.double() - y).abs() <= tol)[t:, 1].all()
    if where == "v":
        rows = [p for p in range(P) if p != 3]
        assert ((out.double() - y).abs() <= tol)[t:, 0][:, rows].all()
    first = d["slots"][0].item()
    err = (pool[first].double() - want[first]).norm(dim=-1)
    half = 2.0 ** -8 * want[first].norm(dim=-1) if state == torch.bfloat16 else 0.0
    assert (err <= min(250, 1.0 / (1.0 - most)) * 2.0 ** -20 * R[first] + half).all()


def test_broadcast_operands(op):
    """One key and query for all key heads, one decay and gate for all heads, by strides of zero."""
    d = make([100, 40], H=4, G=4, seed=113)
    e = {k: (v.contiguous() if k in ("q", "k") else v) for k, v in d.items()}
    for k in ("q", "k", "dt", "b"):
        d[k] = d[k][:, :1].contiguous().expand_as(d[k])
        e[k] = d[k].contiguous()
    assert d["k"].stride(1) == 0
    check(e, *call(op, d), reference(e))
    pool, out = d["pool"].clone(), torch.zeros_like(d["v"][:2])
    step(op, d, pool, out, slice(0, 2))
    pool2, out2 = d["pool"].clone(), torch.zeros_like(out)
    step(op, e, pool2, out2, slice(0, 2))
    assert torch.equal(pool, pool2) and torch.equal(out, out2)


def test_the_same_bits_beside_other_work(op):
    """Chunks of every SM beside a stream that keeps memory busy: the bits of the call alone, many
    times (a piece of an operand read after its place was given away would show here)."""
    for N, state in ((128, torch.float32), (64, torch.bfloat16)):
        d = make([700, 650, 600, 64, 1], H=32, N=N, G=8, state=state, seed=127)
        want = call(op, d)
        ws = torch.empty(op.delta_workspace_bytes(d["pool"], d["v"], d["k"], d["slots"]),
                         dtype=torch.uint8, device="cuda")
        pools, outs = [d["pool"].clone() for _ in range(20)], []
        side, a = torch.cuda.Stream(), torch.zeros(1 << 26, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(40):
                a.add_(1.0)
        for pool in pools:
            outs.append(torch.full(d["v"].shape, 7.0, dtype=torch.bfloat16, device="cuda"))
            op.delta_prompts(pool, d["slots"], d["cu"], d["q"], d["k"], d["v"], d["dt"],
                             d["dt_bias"], d["A"], d["b"], outs[-1], ws, fresh=d["fresh"])
        torch.cuda.synchronize()
        for out, pool in zip(outs, pools):
            assert torch.equal(out, want[0]) and torch.equal(pool, want[1])


@pytest.mark.parametrize("lens,N", [([1, 1, 1], 128), ([9, 6, 5], 64), ([100, 70], 128),
                                    ([90, 80], 64)], ids=str)
@pytest.mark.parametrize("size", [2.0 ** 65, 2.0 ** 127])
def test_keys_past_fp32_become_zeros(op, lens, N, size):
    """A key whose squares' sum is past fp32, finite itself: its token decays the state and reads it,
    and neither products with it nor with the query (of 4, so that they overflow too) leave a trace.
    One token, few tokens, and chunks."""
    d = make(lens, N=N, seed=131)
    steps = max(lens) == 1
    if steps:
        d["fresh"] = None
    t = d["cu"][1].item() + lens[1] // 2
    d["k"], d["q"] = d["k"].clone(), d["q"].clone()
    d["k"][t, 0], d["q"][t, 0] = size, 4.0
    zeroed = dict(d, k=d["k"].clone())
    zeroed["k"][t, 0] = 0.0
    if steps:
        pool, out = d["pool"].clone(), torch.zeros_like(d["v"])
        step(op, d, pool, out)
        torch.cuda.synchronize()
    else:
        out, pool = call(op, d)
    check(d, out, pool, reference(zeroed), chunked=sum(lens) > 36)
    if sum(lens) > 36:  # in chunks a query's does too: its readout is zero
        d["q"][t, 0] = size
        out, _ = call(op, d)
        assert (out[t, :2] == 0).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("N,H", [(128, 4), (64, 8)])
def test_many_prompts_by_64_bit_indices(op, N, H):
    """The plan of more than 32 prompts from int64 slots and offsets, bad and empty prompts among
    them, rows of no prompt on both sides."""
    lens = [(53 * i) % 150 if i % 7 else 0 for i in range(45)]
    d = make(lens, H=H, N=N, G=2, seed=157, idx=torch.int64, lead=3, gap=5)
    d["slots"][4], d["slots"][30] = len(d["pool"]), -(1 << 40)
    check_some(op, d, skip=(4, 30))


def test_a_workspace_of_a_larger_call(op):
    """One buffer, asked for once with the most prompts and tokens, serves calls of any smaller size,
    in chunks or not, and a call token by token takes none."""
    big = make([20] * 60, H=8, seed=163)
    n = op.delta_workspace_bytes(big["pool"], big["v"], big["k"], big["slots"])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for lens in ([20] * 60, [700], [1, 2, 3], [64] * 3, [33], [1] * 50):
        d = make(lens, H=8, seed=167)
        pool, out = d["pool"].clone(), torch.full(d["v"].shape, 7.0, dtype=torch.bfloat16,
                                                  device="cuda")
        op.delta_prompts(pool, d["slots"], d["cu"], d["q"], d["k"], d["v"], d["dt"], d["dt_bias"],
                         d["A"], d["b"], out, None if sum(lens) < 20 else ws, fresh=d["fresh"])
        torch.cuda.synchronize()
        check(d, out, pool, reference(d))
