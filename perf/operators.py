"""The operators of a hybrid model's token mixers around the decode-step state update, as a
serving loop calls them: prompts through the state-space layer, the queries and keys of an
attention layer on their way into a paged cache, and one new token's attention over that cache.

``run`` computes an operator in its plain form (elementary torch operations in fp32, rounded once
at the end), or, where ``own`` is true, by the library's entry points.  ``exact`` evaluates the
definitions in fp64.  Lengths belong to a case (they follow from its values alone); tensors, page
placement and slots come from the seed.
"""

from __future__ import annotations

import functools
import math
import random

import torch

own = False

HEADDIM = 64      # rows of a state-space head
PLAIN_CHUNK = 64  # tokens per chunk of the plain prompt form

# One call's most work: drawn cases stay at or below the largest listed ones.
MOST_TOKEN_HEADS = 32768 * 64
MOST_ROTATED = 8192 * 48 * 128
MOST_KEYS = 2 * 120_001 * 2 * 128


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # a short continuation of one conversation's state: latency is all that counts
        dict(name="prompt 37", op="prompts", prompts=1, tokens=37, spread=0.0, heads=16, groups=1,
             dstate=128, state="f32", fresh=0.0),
        # one ordinary prompt, from an empty state
        dict(name="prompt 2000", op="prompts", prompts=1, tokens=2000, spread=0.0, heads=16,
             groups=1, dstate=128, state="f32", fresh=1.0),
        # a scheduler's packed batch: many prompts of very different lengths, some continuing
        dict(name="prompts ragged 8192", op="prompts", prompts=24, tokens=8192, spread=1.5,
             heads=16, groups=1, dstate=128, state="f32", fresh=0.7),
        # short state rows kept in bf16, with several groups of B and C
        dict(name="prompts bf16 groups", op="prompts", prompts=6, tokens=5003, spread=0.5,
             heads=32, groups=4, dstate=64, state="bf16", fresh=0.5),
        # the largest call: eight long prompts through every head of an unsharded layer
        dict(name="prompts 8 x 4096", op="prompts", prompts=8, tokens=32768, spread=0.0, heads=64,
             groups=1, dstate=128, state="f32", fresh=1.0),
        # the new tokens of a small decode batch
        dict(name="rotate 8", op="rotate", tokens=8, q_heads=16, kv_heads=2, dim=128, rotary=128,
             interleaved=False, page=16),
        # an odd chunk of a prompt, a quarter of a short head rotated, neighbours paired
        dict(name="rotate 777 pairs", op="rotate", tokens=777, q_heads=8, kv_heads=8, dim=64,
             rotary=16, interleaved=True, page=24),
        # a full prompt batch
        dict(name="rotate 8192", op="rotate", tokens=8192, q_heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, page=16),
        # one user, a short cache: latency
        dict(name="attend 1 x 500", op="attend", requests=1, keys=500, spread=0.0, q_heads=16,
             kv_heads=2, dim=128, page=16, window=0, sinks=0),
        # a full decode batch of very different lengths, among them an empty one
        dict(name="attend 128 ragged", op="attend", requests=128, keys=128 * 600, spread=1.0,
             q_heads=16, kv_heads=2, dim=128, page=16, window=0, sinks=0),
        # two very long caches: little to split over but the length
        dict(name="attend 2 x 120001", op="attend", requests=2, keys=240_002, spread=0.0,
             q_heads=16, kv_heads=2, dim=128, page=64, window=0, sinks=0),
        # a layer that looks at the last 1000 tokens and the first four, one key head per query
        # head, pages of an odd size
        dict(name="attend window", op="attend", requests=40, keys=40 * 3001, spread=0.6, q_heads=8,
             kv_heads=8, dim=64, page=24, window=1000, sinks=4),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n + (n == 3072)))


def draw(rng):
    while True:
        c = _draw(rng)
        if _row(c) != 3072:
            return c


def _row(c):
    """Width of the packed activation that a case's operands are views into."""
    if c["op"] == "prompts":
        return c["heads"] * HEADDIM + 2 * c["groups"] * c["dstate"]
    return (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"]


def _draw(rng):
    op = rng.choice(("prompts", "prompts", "rotate", "attend", "attend"))
    if op == "prompts":
        heads = rng.choice((8, 16, 32, 64))
        tokens = _log_int(rng, 1, min(32768, MOST_TOKEN_HEADS // heads))
        return dict(op=op, prompts=min(tokens, _log_int(rng, 1, 64)), tokens=tokens,
                    spread=round(rng.uniform(0.0, 1.5), 3), heads=heads,
                    groups=rng.choice((1, 1, 2, 4, 8)), dstate=rng.choice((64, 128, 128)),
                    state=rng.choice(("f32", "f32", "bf16")), fresh=round(rng.random(), 3))
    dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    q_heads = kv_heads * rng.choice((1, 2, 4, 8))
    if op == "rotate":
        most = MOST_ROTATED // ((q_heads + 2 * kv_heads) * dim)
        return dict(op=op, tokens=_log_int(rng, 1, min(8192, most)), q_heads=q_heads,
                    kv_heads=kv_heads, dim=dim, rotary=dim // rng.choice((1, 2, 4)),
                    interleaved=rng.random() < 0.5, page=rng.choice((16, 24, 64)))
    requests = _log_int(rng, 1, 160)
    keys = _log_int(rng, requests, MOST_KEYS // (kv_heads * dim))
    windowed = rng.random() < 0.4
    return dict(op=op, requests=requests, keys=keys, spread=round(rng.uniform(0.0, 1.0), 3),
                q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=rng.choice((16, 24, 64)),
                window=_log_int(rng, 1, 5000) if windowed else 0,
                sinks=rng.choice((0, 4, 16)) if windowed else 0)


def _lengths(parts, total, spread):
    """``parts`` lengths adding up to ``total``, log-normally spread (0: even)."""
    rng = random.Random(parts * 1_000_003 + total)
    w = [math.exp(spread * rng.gauss(0.0, 1.0)) for _ in range(parts)]
    cut, at = [0], 0.0
    for x in w:
        at += x
        cut.append(int(round(total * at / sum(w))))
    return [b - a for a, b in zip(cut, cut[1:])]


def _caches(case):
    """Keys of each request; in a batch of more than 8 one cache is still empty."""
    lens = _lengths(case["requests"], case["keys"], case["spread"])
    if len(lens) > 8:
        lens[len(lens) // 2] = 0
    return lens


def _visible(n, window, sinks):
    return n if not window else min(n, window + min(sinks, max(0, n - window)))


def work(case):
    c = case
    if c["op"] == "prompts":
        T, H, N, G, P = c["tokens"], c["heads"], c["dstate"], c["groups"], HEADDIM
        lens = _lengths(c["prompts"], T, c["spread"])
        fresh = _fresh(c)
        size = 4 if c["state"] == "f32" else 2
        reads = sum(not f for f in fresh)
        state = (reads + len(lens)) * H * P * N * size
        tokens = T * (2 * H * P + 2 * G * N + H) * 2
        # the recurrence's own products and sums: decay, outer product and readout of each token
        return {"bytes": tokens + state, "flops": 6 * T * H * P * N}
    if c["op"] == "rotate":
        q, k = c["tokens"] * c["q_heads"] * c["dim"], c["tokens"] * c["kv_heads"] * c["dim"]
        table = c["tokens"] * c["rotary"] * 4
        return {"bytes": 2 * 2 * (q + 2 * k) + table + 16 * c["tokens"], "flops": 8 * (q + k)}
    lens = [_visible(n, c["window"], c["sinks"]) for n in _caches(c)]
    cache = sum(lens) * c["kv_heads"] * c["dim"] * 2 * 2
    ends = 2 * c["requests"] * c["q_heads"] * c["dim"] * 2
    pages = sum(-(-n // c["page"]) for n in lens) * 4
    return {"bytes": cache + ends + pages, "flops": 4 * sum(lens) * c["q_heads"] * c["dim"]}


# ---- inputs --------------------------------------------------------------------------------

def _fresh(case):
    rng = random.Random(case["tokens"] * 31 + case["prompts"])
    return [rng.random() < case["fresh"] for _ in range(case["prompts"])]


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
    s = {"prompts": _prepare_prompts, "rotate": _prepare_rotate,
         "attend": _prepare_attend}[case["op"]](case, g)
    s["case"] = case
    if own:
        s["library"] = _library()
        if case["op"] == "prompts":
            n = s["library"].prompts_workspace_bytes(s["pool"], s["x"], s["B"], s["slots"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        elif case["op"] == "attend":
            n = s["library"].attend_workspace_bytes(s["q"], s["k_pages"])
            s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return s


def _prepare_prompts(c, g):
    T, bs, H, G, N, P = c["tokens"], c["prompts"], c["heads"], c["groups"], c["dstate"], HEADDIM
    lens = _lengths(bs, T, c["spread"])
    cu = torch.tensor([0] + lens).cumsum(0).int()
    # x, B and C are views into the one packed activation that the layer's input product leaves
    xbc = _normal(g, T, H * P + 2 * G * N)
    return dict(
        lens=lens, cu=cu.cuda(), fresh=torch.tensor(_fresh(c), dtype=torch.uint8).cuda(),
        pool=_normal(g, bs + 7, H, P, N,
                     dtype=torch.float32 if c["state"] == "f32" else torch.bfloat16),
        slots=torch.randperm(bs + 7, generator=g, device="cuda")[:bs].int(),
        x=xbc[:, :H * P].view(T, H, P), B=xbc[:, H * P:H * P + G * N].view(T, G, N),
        C=xbc[:, H * P + G * N:].view(T, G, N),
        dt=_uniform(g, -4.0, 0.0, T, H).bfloat16(), dt_bias=_uniform(g, -1.0, 1.0, H),
        A=-torch.exp(_uniform(g, 0.0, math.log(16.0), H)), D=_uniform(g, 0.0, 1.0, H),
        out=torch.zeros(T, H, P, dtype=torch.bfloat16, device="cuda"))


def _rotation_table(positions, rotary):
    freq = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq[None]
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


def _prepare_rotate(c, g):
    T, Hq, Hk, d = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
    pages, places = -(-T // c["page"]) + 5, 8192
    qkv = _normal(g, T, (Hq + 2 * Hk) * d)
    return dict(
        q=qkv[:, :Hq * d].view(T, Hq, d), k=qkv[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d),
        v=qkv[:, (Hq + Hk) * d:].view(T, Hk, d),
        q_weight=_uniform(g, 0.5, 1.5, d), k_weight=_uniform(g, 0.5, 1.5, d),
        table=_rotation_table(places, c["rotary"]),
        positions=torch.randint(0, places, (T,), generator=g, device="cuda", dtype=torch.int32),
        slots=torch.randperm(pages * c["page"], generator=g, device="cuda")[:T].int(),
        k_pages=_normal(g, pages, c["page"], Hk, d), v_pages=_normal(g, pages, c["page"], Hk, d),
        out=torch.zeros(T, Hq, d, dtype=torch.bfloat16, device="cuda"))


def _prepare_attend(c, g):
    bs, Hq, Hk, d, page = c["requests"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    lens = _caches(c)
    most = max(1, -(-max(lens) // page))
    need = sum(-(-n // page) for n in lens)
    order = torch.randperm(need + 9, generator=g, device="cuda").int()
    table = torch.zeros(bs, most, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = order[at:at + k]
        at += k
    return dict(
        lens=lens, lengths=torch.tensor(lens, dtype=torch.int32).cuda(), page_table=table,
        q=_normal(g, bs, Hq, d) * 2, k_pages=_normal(g, need + 9, page, Hk, d),
        v_pages=_normal(g, need + 9, page, Hk, d), scale=d ** -0.5,
        out=torch.zeros(bs, Hq, d, dtype=torch.bfloat16, device="cuda"))


# ---- one pass ------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if c["op"] == "prompts":
        if own:
            s["library"].prompts(s["pool"], s["slots"], s["cu"], s["x"], s["dt"], s["dt_bias"],
                                 s["A"], s["B"], s["C"], s["D"], s["out"], s["workspace"],
                                 fresh=s["fresh"])
        else:
            _plain_prompts(s)
        return {"out": s["out"], "pool": s["pool"]}
    if c["op"] == "rotate":
        if own:
            s["library"].rotate_qk(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"],
                                   s["table"], s["positions"], s["out"], s["k_pages"],
                                   s["v_pages"], s["slots"], eps=1e-6,
                                   interleaved=c["interleaved"])
        else:
            _plain_rotate(s)
        return {"q": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if own:
        s["library"].attend(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["lengths"],
                            s["out"], s["workspace"], scale=s["scale"], window=c["window"],
                            sinks=c["sinks"])
    else:
        _plain_attend(s)
    return s["out"]


def _segment_sums(a):
    """L[..., i, j] = a[j+1] + ... + a[i] for j <= i, -inf above the diagonal."""
    n = a.shape[-1]
    i = torch.arange(n, device=a.device)
    low = a[..., :, None].expand(*a.shape, n).masked_fill(i[:, None] <= i[None], 0.0)
    return low.cumsum(-2).masked_fill(i[:, None] < i[None], -math.inf)


def _plain_prompts(s):
    """Chunks of every prompt, padded to PLAIN_CHUNK tokens whose dt is 0 (a step that changes
    nothing); inside a chunk one masked matrix product, between chunks the states' recurrence
    as a product with the matrix of its decays."""
    Q, dev = PLAIN_CHUNK, s["x"].device
    lens = torch.tensor(s["lens"])
    T, H, P = s["x"].shape
    G, N = s["B"].shape[1:]
    # chunk k belongs to prompt who[k], is its nth[k]-th and starts at token first[k]
    per = (lens + Q - 1) // Q
    who = torch.repeat_interleave(torch.arange(len(per)), per)
    nth = torch.arange(len(who)) - (per.cumsum(0) - per)[who]
    at = (lens.cumsum(0) - lens)[who][:, None] + nth[:, None] * Q + torch.arange(Q)
    live = nth[:, None] * Q + torch.arange(Q) < lens[who][:, None]
    at = torch.where(live, at, 0).to(dev, non_blocking=True)
    live, who, nth = (t.to(dev, non_blocking=True) for t in (live, who, nth))
    x = s["x"][at].float() * live[..., None, None]                       # [k, Q, H, P]
    B, C = (t[at].float().repeat_interleave(H // G, 2) for t in (s["B"], s["C"]))
    z = s["dt"][at].float() + s["dt_bias"]
    dt = torch.where(z > 20.0, z, torch.log1p(torch.exp(z))) * live[..., None]
    a = (dt * s["A"]).movedim(-1, 1)                                     # [k, H, Q]
    decay = torch.exp(_segment_sums(a))                                  # [k, H, i, j]
    xdt = (x * dt[..., None]).movedim(2, 1)                              # [k, H, Q, P]
    B, C = B.movedim(2, 1), C.movedim(2, 1)                              # [k, H, Q, N]
    y = (torch.matmul(C, B.transpose(-1, -2)) * decay) @ xdt
    local = (xdt * decay[..., -1, :, None]).transpose(-1, -2) @ B        # [k, H, P, N]
    # states before each chunk and after the last: per prompt over its chunks, element 0 the
    # state that the prompt begins from
    bs, most = len(s["lens"]), int(per.max())
    slots = s["slots"].long()
    start = s["pool"][slots].float()
    start = torch.where((s["fresh"] != 0)[:, None, None, None], torch.zeros_like(start), start)
    chain = torch.zeros(bs, most + 1, H, P * N, device=dev)
    chain[:, 0] = start.flatten(2)
    chain[who, nth + 1] = local.flatten(2)
    total = torch.zeros(bs, most + 1, H, device=dev)
    total[who, nth + 1] = a.sum(-1)
    weight = torch.exp(_segment_sums(total.movedim(-1, 1)))              # [bs, H, z, c]
    after = torch.matmul(weight, chain.movedim(2, 1))                    # [bs, H, z, P N]
    before = after[who, :, nth].view(-1, H, P, N)
    y = y + torch.exp(a.cumsum(-1))[..., None] * (C @ before.transpose(-1, -2))
    y = y.movedim(1, 2) + s["D"][:, None] * x
    # padded tokens land in a spare row
    to = torch.where(live, at, T)
    out = torch.empty(T + 1, H, P, dtype=torch.bfloat16, device=dev)
    out[to] = y.bfloat16()
    s["out"].copy_(out[:T])
    s["pool"][slots] = after[:, :, -1].view(bs, H, P, N).to(s["pool"].dtype)


def _plain_rotate(s):
    half = s["table"].shape[1] // 2
    places = s["positions"].long()
    cos, sin = (t[:, None] for t in s["table"][places].split(half, 1))

    def turn(t, weight):
        t = t.float()
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * weight
        if s["case"]["interleaved"]:
            a, b = t[..., 0:2 * half:2], t[..., 1:2 * half:2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = t[..., :half], t[..., half:2 * half]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, t[..., 2 * half:]], -1).bfloat16()

    slots = s["slots"].long()
    s["out"].copy_(turn(s["q"], s["q_weight"]))
    s["k_pages"].view(-1, *s["k"].shape[1:])[slots] = turn(s["k"], s["k_weight"])
    s["v_pages"].view(-1, *s["v"].shape[1:])[slots] = s["v"]


def _plain_attend(s):
    c = s["case"]
    bs, Hq, d = s["q"].shape
    Hk, page = c["kv_heads"], c["page"]
    most = s["page_table"].shape[1] * page
    k, v = (t[s["page_table"].long()].view(bs, most, Hk, d).float().movedim(2, 1)
            for t in (s["k_pages"], s["v_pages"]))                       # [bs, Hk, keys, d]
    q = s["q"].float().view(bs, Hk, Hq // Hk, d)
    at = torch.arange(most, device=q.device)
    n = s["lengths"][:, None]
    seen = at < n
    if c["window"]:
        seen = seen & ((at >= n - c["window"]) | (at < c["sinks"]))
    seen = seen[:, None, None]
    score = (q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(o.view(bs, Hq, d))


# ---- the definitions in fp64 ---------------------------------------------------------------

def exact(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "prompts":
        return _exact_prompts(case, _prepare_prompts(case, g))
    if case["op"] == "rotate":
        return _exact_rotate(case, _prepare_rotate(case, g))
    return _exact_attend(case, _prepare_attend(case, g))


def _exact_prompts(case, s):
    """Token by token: S <- S exp(dt A) + dt x (x) B,  y = S C + D x."""
    lens, slots = s["lens"], s["slots"].long()
    H, G = case["heads"], case["groups"]
    group = torch.arange(H, device="cuda") // (H // G)
    S = s["pool"].double()[slots]
    S[s["fresh"] != 0] = 0.0
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dt = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=700.0)
    dA = torch.exp(dt * s["A"].double())
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    S = S[torch.tensor(order, device="cuda")]  # longest first: the first m are the live ones
    first = (s["cu"].long()[:-1])[torch.tensor(order, device="cuda")]
    m = len(order)
    for t in range(max(lens)):
        while m and lens[order[m - 1]] <= t:
            m -= 1
        row = first[:m] + t
        x, B, C = (s[n][row].double() for n in ("x", "B", "C"))
        live = S[:m]
        live.mul_(dA[row][..., None, None])
        live.addcmul_((x * dt[row][..., None])[..., None], B[:, group][:, :, None])
        y[row] = torch.matmul(live, C[:, group][..., None])[..., 0] + s["D"].double()[:, None] * x
    pool = s["pool"].double()
    pool[slots[torch.tensor(order, device="cuda")]] = S
    return {"out": y, "pool": pool}


def _exact_rotate(case, s):
    half = case["rotary"] // 2
    angle = s["table"].double()[s["positions"].long()]

    def turn(t, weight):
        t = t.double()
        t = t / torch.sqrt((t * t).sum(-1, keepdim=True) / t.shape[-1] + 1e-6) * weight.double()
        i = torch.arange(half, device="cuda")
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        z = torch.complex(t[..., lo], t[..., hi]) \
            * torch.complex(angle[:, None, :half], angle[:, None, half:])
        t = t.clone()
        t[..., lo], t[..., hi] = z.real, z.imag
        return t

    k, v, slots = s["k_pages"].double(), s["v_pages"].double(), s["slots"].long()
    page = slots // case["page"], slots % case["page"]
    k[page] = turn(s["k"], s["k_weight"])
    v[page] = s["v"].double()
    return {"q": turn(s["q"], s["q_weight"]), "k_pages": k, "v_pages": v}


def _exact_attend(case, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    share = case["q_heads"] // case["kv_heads"]
    for b, n in enumerate(s["lens"]):
        if n == 0:
            continue
        pages = s["page_table"][b, :-(-n // case["page"])].long()
        keep = torch.arange(n, device="cuda")
        if case["window"]:
            keep = keep[(keep >= n - case["window"]) | (keep < case["sinks"])]
        k, v = (t[pages].flatten(0, 1)[keep].double().repeat_interleave(share, 1)
                for t in (s["k_pages"], s["v_pages"]))
        p = torch.softmax(torch.einsum("hd,nhd->hn", s["q"][b].double(), k) * s["scale"], 1)
        out[b] = torch.einsum("hn,nhd->hd", p, v)
    return out
