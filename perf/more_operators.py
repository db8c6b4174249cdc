"""Operators of a hybrid model's delta-rule layers: the gated delta rule for one new token per
request and for packed prompts, over a pool of states, and the residual addition with RMS norm
that stands before every layer, with an output in bf16 or in 8 bits with scales.

``run`` computes an operator in its plain form (elementary torch operations in fp32, rounded once
at the end), or, where ``own`` is true, by the library's entry points.  ``exact`` evaluates the
definitions in fp64.  Lengths belong to a case (they follow from its values alone); tensors and
slots come from the seed.
"""

from __future__ import annotations

import functools
import math
import random

import torch

own = False

PLAIN_CHUNK = 64  # tokens per chunk of the plain prompt form
EPS = 1e-6
E4M3_MOST = 448.0

# One call's most work: drawn cases stay at or below the largest listed ones.
MOST_STEP = 256 * 32 * 128 * 128          # state elements of a decode step
MOST_PROMPT = 32768 * 32 * 128 * 128      # tokens times state elements
MOST_NORM = 16384 * 8192                  # elements of a residual


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one user's new token: latency is all that counts
        dict(name="delta step 1", op="step", requests=1, heads=32, groups=16, headdim=128,
             dstate=128, state="f32"),
        # an odd batch through short rows kept in bf16
        dict(name="delta step 61 bf16", op="step", requests=61, heads=16, groups=8, headdim=64,
             dstate=64, state="bf16"),
        # a full decode batch
        dict(name="delta step 256", op="step", requests=256, heads=32, groups=16, headdim=128,
             dstate=128, state="f32"),
        # a short continuation of one conversation's state
        dict(name="delta prompt 37", op="prompts", prompts=1, tokens=37, spread=0.0, heads=32,
             groups=16, headdim=128, dstate=128, state="f32", fresh=0.0),
        # one ordinary prompt, from an empty state
        dict(name="delta prompt 2000", op="prompts", prompts=1, tokens=2000, spread=0.0, heads=32,
             groups=16, headdim=128, dstate=128, state="f32", fresh=1.0),
        # a scheduler's packed batch: many prompts of very different lengths, some continuing
        dict(name="delta prompts ragged 8192", op="prompts", prompts=24, tokens=8192, spread=1.5,
             heads=16, groups=8, headdim=128, dstate=128, state="f32", fresh=0.7),
        # short heads and state rows in bf16, several heads to a key head
        dict(name="delta prompts bf16 groups", op="prompts", prompts=6, tokens=5003, spread=0.5,
             heads=32, groups=4, headdim=64, dstate=64, state="bf16", fresh=0.5),
        # the largest call: eight long prompts through every head of an unsharded layer
        dict(name="delta prompts 8 x 4096", op="prompts", prompts=8, tokens=32768, spread=0.0,
             heads=32, groups=16, headdim=128, dstate=128, state="f32", fresh=1.0),
        # the new tokens of a small decode batch
        dict(name="norm 8", op="norm", tokens=8, width=4096, residual="bf16", out="bf16", group=0),
        # an odd chunk of a prompt into an 8-bit product, one scale to a row
        dict(name="norm 777 e4m3 rows", op="norm", tokens=777, width=2560, residual="f32",
             out="e4m3", group=2560),
        # a prompt batch into an 8-bit product with scales of 128 columns
        dict(name="norm 8192 e4m3", op="norm", tokens=8192, width=4096, residual="bf16",
             out="e4m3", group=128),
        # the largest prompt batch through a wide model
        dict(name="norm 16384", op="norm", tokens=16384, width=8192, residual="bf16", out="bf16",
             group=0),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n))


def draw(rng):
    op = rng.choice(("step", "prompts", "prompts", "norm"))
    if op == "norm":
        width = 8 * _log_int(rng, 8, 1024)
        out = rng.choice(("bf16", "e4m3"))
        group = 0
        if out == "e4m3":
            group = rng.choice((width, 64, 128))
            width = -(-width // group) * group if group != width else width
        return dict(op=op, tokens=_log_int(rng, 1, MOST_NORM // max(width, 8192)), width=width,
                    residual=rng.choice(("bf16", "bf16", "f32", "none")), out=out, group=group)
    heads = rng.choice((8, 16, 32))
    c = dict(op=op, heads=heads, groups=heads // rng.choice((1, 2, 4)),
             headdim=rng.choice((64, 128, 128)), dstate=rng.choice((64, 128, 128)),
             state=rng.choice(("f32", "f32", "bf16")))
    size = heads * c["headdim"] * c["dstate"]
    if op == "step":
        return dict(c, requests=_log_int(rng, 1, min(512, MOST_STEP // size)))
    tokens = _log_int(rng, 1, min(32768, MOST_PROMPT // size))
    return dict(c, prompts=min(tokens, _log_int(rng, 1, 64)), tokens=tokens,
                spread=round(rng.uniform(0.0, 1.5), 3), fresh=round(rng.random(), 3))


def _lengths(parts, total, spread):
    """``parts`` lengths adding up to ``total``, log-normally spread (0: even)."""
    rng = random.Random(parts * 1_000_003 + total)
    w = [math.exp(spread * rng.gauss(0.0, 1.0)) for _ in range(parts)]
    cut, at = [0], 0.0
    for x in w:
        at += x
        cut.append(int(round(total * at / sum(w))))
    return [b - a for a, b in zip(cut, cut[1:])]


def _fresh(case):
    rng = random.Random(case["tokens"] * 31 + case["prompts"])
    return [rng.random() < case["fresh"] for _ in range(case["prompts"])]


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["tokens"] * c["width"]
        residual = {"bf16": 2 * 2, "f32": 2 * 4, "none": 0}[c["residual"]]
        out = 2 if c["out"] == "bf16" else 1
        scales = 4 * (n // c["group"]) if c["group"] else 0
        return {"bytes": n * (2 + residual + out) + scales + 4 * c["width"], "flops": 5 * n}
    H, G, P, N = c["heads"], c["groups"], c["headdim"], c["dstate"]
    size = 4 if c["state"] == "f32" else 2
    if c["op"] == "step":
        tokens, states = c["requests"], 2 * c["requests"]
    else:
        tokens = c["tokens"]
        states = sum(not f for f in _fresh(c)) + c["prompts"]
    rows = tokens * (2 * H * P + 2 * G * N + 2 * H) * 2
    # the recurrence's own products and sums: decay, prediction, outer product, readout
    return {"bytes": rows + states * H * P * N * size, "flops": 7 * tokens * H * P * N}


# ---- inputs --------------------------------------------------------------------------------

def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _uniform(g, lo, hi, *shape):
    return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo


@functools.lru_cache(maxsize=None)
def _library():
    """The one handle that a program keeps."""
    import selective_state_update_02_gb300 as ssu
    return ssu.SelectiveStateUpdate(0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = _inputs(case, g)
    s["case"] = case
    if own:
        s["library"] = _library()
        if case["op"] == "prompts":
            n = s["library"].delta_workspace_bytes(s["pool"], s["v"], s["k"], s["slots"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


def _inputs(case, g):
    return _norm_inputs(case, g) if case["op"] == "norm" else _delta_inputs(case, g)


def _delta_inputs(c, g):
    H, G, P, N = c["heads"], c["groups"], c["headdim"], c["dstate"]
    if c["op"] == "step":
        bs = T = c["requests"]
        s = {}
    else:
        bs, T = c["prompts"], c["tokens"]
        lens = _lengths(bs, T, c["spread"])
        s = dict(lens=lens, cu=torch.tensor([0] + lens).cumsum(0).int().cuda(),
                 fresh=torch.tensor(_fresh(c), dtype=torch.uint8).cuda())
    # q, k and v are views into the one packed activation that the layer's short convolution and
    # its silu leave: keys of a head have a common part
    raw = _normal(g, T, 2 * G * N + H * P, dtype=torch.float32)
    qkv = (raw / (1.0 + torch.exp(-raw))).bfloat16()
    pool = 0.1 * _normal(g, bs + 7, H, P, N, dtype=torch.float32)
    s.update(
        pool=pool if c["state"] == "f32" else pool.bfloat16(),
        slots=torch.randperm(bs + 7, generator=g, device="cuda")[:bs].int(),
        q=qkv[:, :G * N].view(T, G, N), k=qkv[:, G * N:2 * G * N].view(T, G, N),
        v=qkv[:, 2 * G * N:].view(T, H, P),
        dt=_uniform(g, -4.0, 0.0, T, H).bfloat16(), dt_bias=_uniform(g, -1.0, 1.0, H),
        A=-torch.exp(_uniform(g, 0.0, math.log(16.0), H)), b=_normal(g, T, H),
        scale=N ** -0.5, out=torch.zeros(T, H, P, dtype=torch.bfloat16, device="cuda"))
    return s


def _norm_inputs(c, g):
    T, W = c["tokens"], c["width"]
    s = dict(x=_normal(g, T, W), weight=_uniform(g, 0.5, 1.5, W), residual=None, scales=None)
    if c["residual"] != "none":
        r = 4.0 * _normal(g, T, W, dtype=torch.float32)
        s["residual"] = r if c["residual"] == "f32" else r.bfloat16()
    if c["out"] == "e4m3":
        s["out"] = torch.zeros(T, W, dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.zeros(T, W // c["group"], device="cuda")
    else:
        s["out"] = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "norm":
        if own:
            s["library"].add_norm(s["x"], s["weight"], s["out"], residual=s["residual"],
                                  scales=s["scales"], eps=EPS)
        else:
            _plain_norm(s)
        return {n: s[n] for n in ("out", "residual", "scales") if s[n] is not None}
    if own:
        if op == "step":
            s["library"].delta(s["pool"], s["slots"], s["q"], s["k"], s["v"], s["dt"],
                               s["dt_bias"], s["A"], s["b"], s["out"], scale=s["scale"],
                               qk_eps=EPS)
        else:
            s["library"].delta_prompts(s["pool"], s["slots"], s["cu"], s["q"], s["k"], s["v"],
                                       s["dt"], s["dt_bias"], s["A"], s["b"], s["out"],
                                       s["workspace"], fresh=s["fresh"], scale=s["scale"],
                                       qk_eps=EPS)
    elif op == "step":
        _plain_step(s)
    else:
        _plain_prompts(s)
    return {"out": s["out"], "pool": s["pool"]}


def _plain_norm(s):
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
        s["residual"].copy_(r)
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["scales"] is None:
        s["out"].copy_(y)
        return
    parts = y.view(y.shape[0], s["scales"].shape[1], -1)
    scale = (parts.abs().amax(-1) / E4M3_MOST).clamp_min(2.0 ** -126)
    s["scales"].copy_(scale)
    s["out"].copy_((parts / scale[..., None]).view_as(y))


def _unit(t, heads):
    """The rows of q or k at length one, a copy for every head that reads them."""
    t = t.float()
    t = t * torch.rsqrt(t.square().sum(-1, keepdim=True) + EPS)
    return t.repeat_interleave(heads // t.shape[-2], -2)


def _rates(s):
    """The log of every token's decay, and beta."""
    z = s["dt"].float() + s["dt_bias"]
    dt = torch.where(z > 20.0, z, torch.log1p(torch.exp(z)))
    return dt * s["A"], 1.0 / (1.0 + torch.exp(-s["b"].float()))


def _plain_step(s):
    slots, heads = s["slots"].long(), s["v"].shape[1]
    q, k = _unit(s["q"], heads) * s["scale"], _unit(s["k"], heads)
    log_a, beta = _rates(s)
    S = s["pool"][slots].float() * torch.exp(log_a)[..., None, None]
    e = beta[..., None] * (s["v"].float() - (S * k[:, :, None]).sum(-1))
    S = S + e[..., None] * k[:, :, None]
    s["out"].copy_((S * q[:, :, None]).sum(-1))
    s["pool"][slots] = S.to(s["pool"].dtype)


def _inverse(L):
    """(I + L)^-1 of strictly lower triangular L, by blocks of twice the size at a time."""
    n = L.shape[-1]
    at = torch.arange(n, device=L.device)
    T = torch.eye(n, device=L.device).expand_as(L)
    size = 1
    while size < n:
        block = at // size
        below = (block[:, None] == block[None] + 1) & (block[:, None] % 2 == 1)
        T = T - T @ (L * below) @ T
        size *= 2
    return T


def _plain_prompts(s):
    """Chunks of every prompt, padded to PLAIN_CHUNK tokens of beta and log decay 0 (a step that
    changes nothing).  A chunk's corrections solve a triangular system; the state goes from
    chunk to chunk, all prompts' n-th chunks at a time."""
    Q, dev = PLAIN_CHUNK, s["v"].device
    lens = torch.tensor(s["lens"])
    T, H, P = s["v"].shape
    slots = s["slots"].long()
    most = max(1, int((lens.max() + Q - 1) // Q))
    first = lens.cumsum(0) - lens
    at = torch.arange(most * Q)[None].expand(len(lens), -1)
    live = at < lens[:, None]
    at = torch.where(live, at + first[:, None], 0).to(dev).view(len(lens), most, Q)
    live = live.to(dev).view(len(lens), most, Q)
    log_a, beta = _rates(s)
    S = s["pool"][slots].float()
    S = torch.where((s["fresh"] != 0)[:, None, None, None], torch.zeros_like(S), S)
    out = torch.empty(T + 1, H, P, dtype=torch.bfloat16, device=dev)  # padding to a spare row
    i = torch.arange(Q, device=dev)
    for n in range(most):
        row, on = at[:, n], live[:, n]
        k = (_unit(s["k"][row], H) * on[..., None, None]).movedim(2, 1)   # [b, H, Q, N]
        q = (_unit(s["q"][row], H) * s["scale"]).movedim(2, 1)
        v = (s["v"][row].float() * on[..., None, None]).movedim(2, 1)
        bt = (beta[row] * on[..., None]).movedim(2, 1)[..., None]         # [b, H, Q, 1]
        total = (log_a[row].double() * on[..., None]).movedim(2, 1).cumsum(-1)
        gap = (total[..., :, None] - total[..., None, :]).float()
        decay = torch.exp(gap.masked_fill(i[:, None] < i[None], -math.inf))
        passed = torch.exp(total).float()[..., None]
        gram = (k @ k.transpose(-1, -2)) * decay
        solve = _inverse(bt * gram * (i[:, None] > i[None]))
        u = solve @ (bt * (v - passed * (k @ S.transpose(-1, -2))))
        y = passed * (q @ S.transpose(-1, -2)) + (q @ k.transpose(-1, -2) * decay) @ u
        S = passed[..., -1:, :] * S + (u * decay[..., -1, :, None]).transpose(-1, -2) @ k
        out[torch.where(on, row, T)] = y.movedim(1, 2).bfloat16()
    s["out"].copy_(out[:T])
    s["pool"][slots] = S.to(s["pool"].dtype)


# ---- the definitions in fp64 ---------------------------------------------------------------

def exact(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = _inputs(case, g)
    return _exact_norm(case, s) if case["op"] == "norm" else _exact_delta(case, s)


def _exact_norm(case, s):
    r = s["x"].double()
    if s["residual"] is not None:
        r = r + s["residual"].double()
    y = r / torch.sqrt((r * r).sum(-1, keepdim=True) / case["width"] + EPS) * s["weight"].double()
    if case["out"] == "bf16":
        return {"out": y} if s["residual"] is None else {"out": y, "residual": r}
    part = y.reshape(case["tokens"], -1, case["group"])
    scale = part.abs().max(-1).values / E4M3_MOST
    answer = {"out": (part / scale[..., None]).reshape(y.shape), "residual": r, "scales": scale}
    if s["residual"] is None:
        del answer["residual"]
    return answer


def _exact_delta(case, s):
    """Token by token: S <- a S,  S <- S + beta (v - S k) (x) k,  y = S q."""
    heads, groups = case["heads"], case["groups"]
    of = torch.arange(heads, device="cuda") // (heads // groups)

    def unit(t):
        t = t.double()
        return (t / torch.sqrt((t * t).sum(-1, keepdim=True) + EPS))[:, of]

    lens = s["lens"] if "lens" in s else [1] * case["requests"]
    slots = s["slots"].long()
    order = torch.tensor(sorted(range(len(lens)), key=lambda b: -lens[b]), device="cuda")
    by_length = sorted(lens, reverse=True)
    first = torch.tensor([0] + lens, device="cuda").cumsum(0)[order]
    S = s["pool"].double()[slots[order]]
    if "fresh" in s:
        S[s["fresh"][order] != 0] = 0.0
    q, k = unit(s["q"]) * s["scale"], unit(s["k"])
    z = s["dt"].double() + s["dt_bias"].double()
    a = torch.exp(torch.nn.functional.softplus(z, threshold=700.0) * s["A"].double())
    beta = torch.sigmoid(s["b"].double())
    y = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    m = len(lens)  # longest first: the first m are the live ones
    for t in range(by_length[0]):
        while m and by_length[m - 1] <= t:
            m -= 1
        row, live = first[:m] + t, S[:m]
        live.mul_(a[row][..., None, None])
        e = s["v"][row].double() - torch.matmul(live, k[row][..., None])[..., 0]
        live.addcmul_((beta[row][..., None] * e)[..., None], k[row][:, :, None])
        y[row] = torch.matmul(live, q[row][..., None])[..., 0]
    pool = s["pool"].double()
    pool[slots[order]] = S
    return {"out": y, "pool": pool}
