"""One token's attention over the paged cache (``ssu_attend``) against the definition in fp64.

Tolerance, derived before any run.  With p the exact weights and W = sum_j p_j |v_j|: scores of
D products in fp32 are off by at most (D + 4) 2^-24 sum |q k| scale <= 2^-13 here, so a weight by
2^-12.9 of itself (numerator and normaliser: 2^-11.9), its exponential by 2^-21, its rounding to
bf16 by 2^-8, and partial sums by a few 2^-24.  An output is within 2^-8 |o| + (2^-8 + 2^-11) W.
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


def make(lens, Hq=4, Hk=2, D=128, page=16, seed=0, idx=torch.int32, spare=3, more=0):
    g = torch.Generator().manual_seed(seed)
    bs = len(lens)
    most = max([-(-n // page) for n in lens] + [0]) + more
    need = sum(-(-n // page) for n in lens)
    order = torch.randperm(need + spare, generator=g)
    table = torch.full((bs, most), -7, dtype=torch.int64)  # columns past a length are not read
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = order[at:at + k]
        at += k
    return dict(
        q=(torch.randn(bs, Hq, D, generator=g) * 2).bfloat16().cuda(),
        k_pages=torch.randn(need + spare, page, Hk, D, generator=g).bfloat16().cuda(),
        v_pages=torch.randn(need + spare, page, Hk, D, generator=g).bfloat16().cuda(),
        page_table=table.to(idx).cuda(), lengths=torch.tensor(lens).to(idx).cuda(),
        out=torch.full((bs, Hq, D), 7.0, dtype=torch.bfloat16).cuda())


def reference(d, scale=None, window=0, sinks=0, drop=()):
    """(o, W) in fp64; ``drop``: (request, page column) pairs that are left out."""
    q, table, lens = d["q"].double(), d["page_table"].tolist(), d["lengths"].tolist()
    bs, Hq, D = q.shape
    page, Hk = d["k_pages"].shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    o = torch.zeros(bs, Hq, D, dtype=torch.float64, device="cuda")
    W = torch.zeros_like(o)
    for b, n in enumerate(lens):
        j = torch.arange(max(n, 0))
        if window:
            j = j[(j >= n - window) | (j < sinks)]
        j = j[[(b, c) not in drop for c in (j // page).tolist()]] if drop else j
        if not len(j):
            continue
        pages = torch.tensor(table[b])[j // page].cuda()
        k, v = (t[pages, (j % page).cuda()].double().repeat_interleave(Hq // Hk, 1)
                for t in (d["k_pages"], d["v_pages"]))
        p = torch.softmax(torch.einsum("hd,nhd->hn", q[b], k) * scale, 1)
        o[b] = torch.einsum("hn,nhd->hd", p, v)
        W[b] = torch.einsum("hn,nhd->hd", p, v.abs())
    return o, W


_WORKSPACES: dict = {}


def workspace(op, d):
    """One workspace for all calls, as a program keeps it: zero once, never cleared again."""
    n = op.attend_workspace_bytes(d["q"], d["k_pages"])
    if n > _WORKSPACES.get("n", 0):
        _WORKSPACES.update(n=n, t=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    return _WORKSPACES.get("t")


def check(got, ref, rows=slice(None)):
    o, W = ref
    err = (got.double() - o)[rows].abs()
    tol = (2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -11) * W)[rows]
    assert (err <= tol).all(), f"off by {(err / tol.clamp_min(1e-300)).max():.3g} of the tolerance"


def run_and_check(op, d, **kw):
    op.attend(**d, workspace=workspace(op, d), **kw)
    torch.cuda.synchronize()
    check(d["out"], reference(d, **kw))


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 1000, 5000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths(op, n, D):
    run_and_check(op, make([n], D=D, seed=n + D))


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 1), (8, 8), (16, 2), (7, 1), (24, 2), (32, 1),
                                   (40, 2), (64, 1), (5, 5)])
def test_heads(op, Hq, Hk):
    run_and_check(op, make([200, 33, 0, 70], Hq, Hk, seed=Hq * 100 + Hk))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 256, 1000])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(op, page, D):
    run_and_check(op, make([500, 1, 999, 64], D=D, page=page, seed=page, more=2))


@pytest.mark.parametrize("idx", [torch.int32, torch.int64], ids=["i32", "i64"])
def test_many_ragged_requests(op, idx):
    lens = [(37 * i * i) % 700 for i in range(300)] + [9000, 0, 1]
    run_and_check(op, make(lens, Hq=8, Hk=2, D=64, seed=1, idx=idx))


def test_one_long_cache(op):
    """One key head: the length is all there is to split over."""
    run_and_check(op, make([40_007], Hq=4, Hk=1, page=64, seed=2))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (100, 16), (64, 64),
                                          (130, 200), (1000, 3), (5000, 5000)])
@pytest.mark.parametrize("page", [16, 24])
def test_window_and_sinks(op, window, sinks, page):
    d = make([0, 1, 15, 99, 100, 101, 116, 117, 130, 700, 4001], Hq=4, Hk=2, page=page,
             seed=window + sinks)
    run_and_check(op, d, window=window, sinks=sinks)


def test_masked_places_are_not_read(op):
    """NaN and infinities past a length, outside the window, and in pages of nobody stay out;
    so do page ids that no visible position uses."""
    d = make([70, 200, 5], page=16, seed=3)
    for t in (d["k_pages"], d["v_pages"]):
        used = torch.zeros(t.shape[:2], dtype=torch.bool)
        for b, n in enumerate((70, 200, 5)):
            for j in range(n):
                if j >= n - 50 or j < 4:
                    used[d["page_table"][b, j // 16], j % 16] = True
        t[~used.cuda()] = float("nan")
    d["page_table"][1, 3] = 10 ** 6  # positions 48 .. 63 lie before the window of 50
    op.get_error()
    run_and_check(op, d, window=50, sinks=4)
    assert op.get_error() == (0, -1)


def test_large_scores(op):
    """Scores far apart: one key takes all the weight; ties share it."""
    d = make([300, 40], seed=4)
    d["q"] *= 50
    op.attend(**d, workspace=workspace(op, d))
    torch.cuda.synchronize()
    # scores of up to 2^13 are off by 2^-24 (D + 4) of their terms' magnitude, below 2^-4, so
    # only near ties can differ: compare where the largest weight is clear of the others
    o, W = reference(d)
    k = d["k_pages"]
    assert torch.isfinite(d["out"].double()).all()
    assert ((d["out"].double() - o).abs() <= 2.0 ** -3 * W + 2.0 ** -8 * o.abs()).all()
    d = make([64], Hq=2, Hk=1, seed=5)
    d["k_pages"][:] = d["k_pages"][0, 0, 0]
    run_and_check(op, d)


def test_infinite_scores_as_weights_of_zero(op):
    """Keys whose score is -inf have no weight, as long as one finite score is there."""
    d = make([100], Hq=2, Hk=1, D=64, seed=6)
    d["q"].fill_(1.0)
    row = d["page_table"][0, 2].item()
    d["k_pages"][row, 3:9] = float("-inf")
    op.attend(**d, workspace=workspace(op, d))
    torch.cuda.synchronize()
    assert torch.isfinite(d["out"].double()).all()
    check(d["out"], reference(d))


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25])
def test_scales(op, scale):
    d = make([90, 3], seed=7)
    d["q"] *= 0.25
    run_and_check(op, d, scale=scale)


def test_strides(op):
    d = make([130, 77], Hq=4, Hk=2, D=64, seed=8)
    n, page = d["k_pages"].shape[:2]
    both = torch.randn(n, 2, 2, page, 80, device="cuda").bfloat16()
    d["k_pages"] = both[:, 0, :, :, :64].transpose(1, 2)   # heads outside rows
    d["v_pages"] = both[:, 1, :, :, 16:].transpose(1, 2)
    d["q"] = torch.randn(2, 6, 72, device="cuda").bfloat16()[:, 1:5, 8:]
    d["out"] = torch.full((2, 5, 64), 7.0, device="cuda").bfloat16()[:, :4]
    d["page_table"] = d["page_table"].t().contiguous().t()
    d["lengths"] = d["lengths"].repeat_interleave(2)[::2]
    run_and_check(op, d)


def test_shared_pages(op):
    """Requests that share a prefix's pages."""
    d = make([160, 160, 100], seed=9)
    d["page_table"][1, :8] = d["page_table"][0, :8]
    d["page_table"][2, :7] = d["page_table"][0, :7]
    run_and_check(op, d)


def test_bad_lengths_and_pages(op):
    d = make([50, 60, 70, 80], seed=10)
    op.get_error()
    d["lengths"][1] = -1
    d["lengths"][2] = d["page_table"].shape[1] * 16 + 1
    d["page_table"][3, 1] = d["k_pages"].shape[0]
    d["page_table"][3, 4] = -1
    op.attend(**d, workspace=workspace(op, d))
    torch.cuda.synchronize()
    ref = {**d, "lengths": torch.tensor([50, 0, 0, 80])}
    check(d["out"], reference(ref, drop=((3, 1), (3, 4))), [0, 3])
    assert (d["out"][1:3] == 7.0).all()
    assert op.get_error() == (4, 1)
    # nothing of a request's cache can be read: zeros, like an empty one
    d["page_table"][:] = -1
    d["lengths"][:] = torch.tensor([50, 1, 0, 80])
    op.attend(**d, workspace=workspace(op, d))
    torch.cuda.synchronize()
    assert (d["out"] == 0).all()
    assert op.get_error() == (4 + 1 + 5, 0)


def test_same_call_same_bits(op):
    d = make([9000, 10, 3000, 0], Hq=8, Hk=1, seed=11)
    op.attend(**d, workspace=workspace(op, d))
    first = d["out"].clone()
    for _ in range(20):
        op.attend(**d, workspace=workspace(op, d))
        assert torch.equal(first, d["out"])


def test_graph_and_side_stream(op):
    d = make([3000, 10, 500], seed=12)
    ws = torch.zeros(op.attend_workspace_bytes(d["q"], d["k_pages"]), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op.attend(**d, workspace=ws, stream=side)
    side.synchronize()
    ref = reference(d)
    check(d["out"], ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.attend(**d, workspace=ws)
    for _ in range(3):
        d["out"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(d["out"], ref)


def test_long_cache_past_32_bit_offsets(op):
    """Pages whose element offsets pass 2^32."""
    d = make([100], Hq=2, Hk=1, D=64, page=16, seed=13)
    n = d["k_pages"].shape[0]
    big = torch.empty((2 ** 32 + 2 ** 20,), dtype=torch.bfloat16, device="cuda")
    far = big[-(n * 16 * 64):].view(n, 16, 1, 64)
    far.copy_(d["k_pages"])
    k = big.as_strided((2 ** 22 + n, 16, 1, 64), (1024, 64, 64, 1))
    base = (big.numel() - n * 1024) // 1024
    assert base * 1024 > 2 ** 32 and base + n <= k.shape[0] + 2 ** 12
    k = big.as_strided((base + n, 16, 1, 64), (1024, 64, 64, 1))
    v = torch.zeros(1, device="cuda").bfloat16()
    ref = reference({**d, "v_pages": d["k_pages"]})
    d["page_table"] += base
    d["k_pages"], d["v_pages"] = k, k
    op.attend(**d, workspace=workspace(op, d))
    torch.cuda.synchronize()
    check(d["out"], ref)


def test_extents_past_32_bits_of_vectors(op):
    """Strides that put a cache's extent past 2^32 16-byte vectors (a single page, so no such
    memory is there)."""
    d = make([60, 13], Hq=4, Hk=2, D=64, page=64, seed=16)
    d["page_table"][1] = d["page_table"][0]
    for k in ("k_pages", "v_pages"):
        one = d[k][int(d["page_table"][0, 0])].clone()
        d[k] = one.as_strided((1, 64, 2, 64), (2 ** 37, 128, 64, 1))
    d["page_table"][:] = 0
    run_and_check(op, d)


def test_no_requests(op):
    d = make([], seed=14)
    d["page_table"] = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    op.attend(**d, workspace=workspace(op, d))
    torch.cuda.synchronize()


def test_refusals(op):
    d = make([40, 50], seed=15)
    ws = torch.zeros(op.attend_workspace_bytes(d["q"], d["k_pages"]), dtype=torch.uint8,
                     device="cuda")

    def attempt(error, **change):
        with pytest.raises(error):
            op.attend(**{**d, "workspace": ws, **change})

    attempt(TypeError, q=d["q"].float())
    attempt(TypeError, lengths=d["lengths"].long())
    attempt(ValueError, out=d["out"][:1])
    attempt(ValueError, v_pages=d["v_pages"][:, :8])
    attempt(ValueError, page_table=d["page_table"][:1])
    attempt(ValueError, lengths=d["lengths"].cpu())
    attempt(ssu.SsuError, q=d["q"][:, :3].contiguous(), out=d["out"][:, :3].contiguous())
    attempt(ssu.SsuError, window=-1)
    attempt(ssu.SsuError, sinks=-1)
    attempt(ssu.SsuError, scale=float("inf"))
    attempt(ssu.SsuError, scale=float("nan"))
    attempt(ssu.SsuError, q=torch.zeros(2, 4, 129, device="cuda").bfloat16()[..., 1:])
    small = torch.zeros(4, 16, 2, 32, device="cuda").bfloat16()
    attempt(ssu.SsuError, k_pages=small, v_pages=small, q=d["q"][..., :32].contiguous(),
            out=d["out"][..., :32].contiguous())
    if ws.numel():
        attempt(ssu.SsuError, workspace=ws[:-256])
        attempt(ssu.SsuError, workspace=None)
    torch.cuda.synchronize()
    assert (d["out"] == 7.0).all() and op.get_error() == (0, -1)
