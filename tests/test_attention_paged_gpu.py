"""attention_paged against a plain loop in 64 bits; every element within a derived bound."""
import math

import numpy as np
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import F8, Step, bound, reference

pytestmark = pytest.mark.gpu

#: A bf16 rounding alone leaves a relative 2-norm error of about 1.65e-3.
RMS = 2.5e-3


def run(step, dev, scale=None, workspace=None, lse=True):
    out_lse = torch.empty(step.T, step.heads, device=dev) if lse else None
    out = dl.attention_paged(step.q.to(dev), step.cache(dev), *step.seqs(dev), max_q=step.max_q,
                             scale=scale, out_lse=out_lse, workspace=workspace)
    torch.cuda.synchronize(dev)
    assert dl.device_status() == 0
    return out, out_lse


def check(step, out, lse, scale=None):
    want, want_lse, spread, biggest = reference(step, scale)
    got = out.double().cpu()
    err = (got - want).abs()
    lim = bound(step, want, spread, biggest)
    assert torch.isfinite(got).all()
    assert (err <= lim).all(), (err / lim).max()
    if want.norm() > 0 and step.T * step.heads * step.dim > 500:
        assert (got - want).norm() / want.norm() < RMS
    if lse is not None:
        a, w = lse.double().cpu(), want_lse
        assert torch.equal(torch.isinf(a), torch.isinf(w))
        fin = torch.isfinite(w)
        assert ((a - w).abs()[fin] <= 1e-4 + 1e-5 * w.abs()[fin]).all()
    return want


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,block", [(8, 8), (16, 4), (32, 1), (64, 16), (128, 128), (256, 32)])
def test_decode_lengths_and_layouts(cuda_device, group, dim, page, block):
    lens = [1, 2, 16, 17, 127, 128, 129, 300]
    step = Step(lens, [1] * len(lens), heads=2 * group, kv_heads=2, dim=dim, page=page, block=block,
                seed=group * 1000 + dim + page)
    check(step, *run(step, cuda_device))


@pytest.mark.parametrize("group,news", [(8, [6, 1, 3, 6]), (8, [16, 16, 2, 9]), (1, [5, 7, 1, 2]), (3, [3, 3, 3, 3]),
                                        (4, [40, 33, 1, 64]), (7, [19, 1, 2, 6]), (5, [13, 4, 9, 1]),
                                        (64, [3, 2, 1, 2]), (128, [2, 1, 1, 1])])
@pytest.mark.parametrize("dim", [64, 128])
def test_several_new_tokens(cuda_device, group, news, dim):
    step = Step([200, 128, 65, 131], news, heads=group, kv_heads=1, dim=dim, page=32, block=8, seed=group)
    check(step, *run(step, cuda_device))


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 15, 16, 17, 24, 25, 31, 33, 40, 47, 48, 49, 57, 64, 65, 80, 96, 111, 127, 128, 129])
def test_every_row_count(cuda_device, rows):
    """One head with `rows` new tokens: each padded row count and its neighbours."""
    step = Step([rows + 30, max(rows // 2, 1) + 150], [rows, max(rows // 2, 1)], heads=1, kv_heads=1,
                page=16, seed=rows)
    check(step, *run(step, cuda_device))


@pytest.mark.parametrize("news", [1, 6])
def test_long_and_split(cuda_device, news):
    """Few sequences of thousands of tokens: the work of one is spread over many CTAs."""
    step = Step([5003, 2048, 777], [news] * 3, heads=8, kv_heads=1, page=64, block=16, seed=21)
    want = check(step, *run(step, cuda_device))
    a, _ = run(step, cuda_device)
    b, _ = run(step, cuda_device, workspace=dl.Workspace(dl.attention_workspace_bytes(
        3, step.T, 8, 1, 128, max_q=news)))
    assert torch.equal(a, b) and want.norm() > 0


def test_many_sequences(cuda_device):
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(1, 90, (700,), generator=g).tolist()
    step = Step(lens, [1] * 700, heads=4, kv_heads=2, dim=64, page=16, seed=22)
    check(step, *run(step, cuda_device))


@pytest.mark.parametrize("most,group", [(4, 8), (6, 8), (8, 8), (3, 3)])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_short_sequences_of_several_tokens(cuda_device, most, group, dim):
    """One CTA goes through several sequences of one or two tiles each: the next one's queries
    follow at once, and some sequences have no new token or see nothing."""
    g = torch.Generator().manual_seed(most)
    news = torch.randint(0, most + 1, (310,), generator=g).tolist()
    lens = [max(n + int(e), 0) for n, e in zip(news, torch.randint(-2, 200, (310,), generator=g))]
    step = Step(lens, news, heads=2 * group, kv_heads=2, dim=dim, page=32, block=8, seed=24)
    check(step, *run(step, cuda_device))


def test_rows_that_see_nothing(cuda_device):
    """No cached tokens, fewer cached than new ones, and only absent pages: zeros."""
    step = Step([0, 3, 40, 150], [2, 5, 1, 4], seed=23)
    step.table[2] = -1
    step.table[3, 1:3] = 10 ** 6
    out, lse = run(step, cuda_device)
    check(step, out, lse)
    assert not out[:4].any() and not out[7].any() and torch.isinf(lse[7]).all()
    none = Step([0, 0], [1, 1], seed=24)
    out, lse = run(none, cuda_device)
    assert not out.any() and (lse == -math.inf).all()


def test_nothing_to_do(cuda_device):
    step = Step([4, 9], [0, 1], seed=25)
    check(step, *run(step, cuda_device))
    empty = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device=cuda_device)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=cuda_device)   # noqa: E731
    assert dl.attention_paged(empty, step.cache(cuda_device), i(0, 1), i(0), i(1), max_q=0).numel() == 0


def test_what_lies_past_the_end_does_not_reach_the_output(cuda_device):
    """NaN codes and NaN scales in unused slots, unused pages and later blocks."""
    for news in (1, 6):
        step = Step([5, 70, 130], [news] * 3, page=64, block=16, seed=26)
        want = reference(step)[0]
        k, v = step.k.view(torch.uint8), step.v.view(torch.uint8)
        used = torch.zeros(step.pages, step.page, dtype=torch.bool)
        for b in range(3):
            for p, o in step.slots(b, step.lens[b]):
                used[p, o] = True
        for x in (k, v):
            x.copy_(torch.where(used[:, None, :, None], x, 127))
        blocks = used.view(step.pages, -1, 16).any(-1)[:, None]
        for x in (step.k_scale, step.v_scale):
            x.copy_(torch.where(blocks, x, float("nan")))
        out, lse = run(step, cuda_device)
        assert torch.isfinite(out).all() and not torch.isnan(lse).any()
        assert (out.double().cpu() - want).norm() / want.norm() < RMS


def test_nan_of_a_later_token_reaches_only_those_that_see_it(cuda_device):
    step = Step([140], [8], heads=8, kv_heads=1, seed=27)
    want = reference(step)[0]
    p, o = step.slots(0, 140)[136]               # new token 4
    step.v.view(torch.uint8)[p, 0, o, 37] = 127
    out, _ = run(step, cuda_device)
    got = out.double().cpu()
    assert torch.isnan(got[4:, :, 37]).all()
    got[4:, :, 37] = want[4:, :, 37]
    assert torch.isfinite(got).all() and (got - want).norm() / want.norm() < RMS
    step.k.view(torch.uint8)[p, 0, o, 5] = 255
    out, _ = run(step, cuda_device)
    assert torch.isnan(out[4:]).all() and torch.isfinite(out[:4]).all()


@pytest.mark.parametrize("news,group", [(1, 8), (2, 8), (3, 8), (6, 8), (8, 8)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("low", [0, 1, 2])
@pytest.mark.parametrize("sequences", [1, 500])
def test_nan_of_a_token_without_weight(cuda_device, news, group, dim, low, sequences):
    """A value that all rows see is NaN; its weight is too small for fp32, and 0 x NaN is NaN
    still, whichever tile it lies in, on a CTA of its own or with the others."""
    step = Step([384], [news], heads=group, kv_heads=1, dim=dim, page=128, block=128, seed=31)
    step.B, step.T = sequences, sequences * news
    step.lens, step.news = [384] * sequences, [news] * sequences
    step.table = step.table.expand(sequences, -1).contiguous()
    step.start = torch.arange(sequences + 1, dtype=torch.int32) * news
    step.q = torch.ones(step.T, group, dim).bfloat16()
    for t in range(3):
        step.k[int(step.table[0, t])] = -16.0 if t == low else 16.0
    step.k_scale.fill_(1)
    step.v_scale.fill_(0.01)
    step.v.view(torch.uint8)[int(step.table[0, low]), 0, 5, 7] = 0x7f
    out, lse = run(step, cuda_device)
    nan = torch.isnan(out.cpu())
    assert nan[:, :, 7].all() and nan.sum() == step.T * group
    assert torch.isfinite(lse).all()


def test_nan_and_infinite_queries(cuda_device):
    step = Step([60, 60], [2, 2], seed=28)
    want = reference(step)[0]
    step.q[1, 3, 8] = float("nan")
    step.q[2, 0, 0] = float("inf")
    out, _ = run(step, cuda_device)
    got = out.double().cpu()
    assert torch.isnan(got[1, 3]).all() and torch.isnan(got[2, 0]).all()
    got[1, 3], got[2, 0] = want[1, 3], want[2, 0]
    assert torch.isfinite(got).all() and (got - want).norm() / want.norm() < RMS


def test_large_and_peaked_scores(cuda_device):
    """Scores of hundreds: one token takes all, and the running maximum keeps moving."""
    step = Step([900, 400], [1, 3], seed=29)
    step.q *= 40
    check(step, *run(step, cuda_device))
    ramp = Step([1000], [1], heads=4, kv_heads=1, seed=30)
    ramp.q = ramp.q.abs()
    for j, (p, o) in enumerate(ramp.slots(0, 1000)):
        ramp.k[p, 0, o] = torch.full((128,), 0.4 * j).clamp(max=448).to(F8)
    ramp.k_scale.fill_(0.01)
    check(ramp, *run(ramp, cuda_device))


def test_scales_that_differ_by_block(cuda_device):
    """Arbitrary fp32 scales, spread over many binades, and blocks of zeros."""
    step = Step([300, 70], [2, 1], block=4, seed=31, pow2=False)
    step.v_scale *= torch.exp(2 * torch.randn(step.v_scale.shape, generator=step.g))
    check(step, *run(step, cuda_device))
    step.v_scale[::2] = 0
    step.k_scale[::3] = 0
    check(step, *run(step, cuda_device))


def test_queries_of_unequal_size(cuda_device):
    """Rows a thousand times apart share a tile, as do large and tiny elements of one row."""
    step = Step([200], [4], heads=8, kv_heads=1, seed=32)
    step.q[:, ::2] *= 30
    step.q[:, 1::2] *= 1 / 32
    step.q[..., 5] *= 20
    check(step, *run(step, cuda_device))


def test_scale_argument(cuda_device):
    step = Step([100], [2], seed=33)
    for s in (0.0, 0.02, 1.0, -0.05):
        check(step, *run(step, cuda_device, scale=s), scale=s)


def test_strided_queries_and_cache_views(cuda_device):
    step = Step([150, 33], [3, 2], seed=34)
    P, H, pg, D = step.k.shape
    big = torch.full((P, 2, 2, H, pg, D), 127, dtype=torch.uint8, device=cuda_device)
    k, v = big[:, 1, 0], big[:, 1, 1]
    k.copy_(step.k.view(torch.uint8))
    v.copy_(step.v.view(torch.uint8))
    sb = torch.full((P, H, 5), float("nan"), device=cuda_device)
    ks, vs = sb[..., 1:2], sb[..., 3:4]
    ks.copy_(step.k_scale)
    vs.copy_(step.v_scale)
    row = torch.full((step.T, 12 * D), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    q = row[:, D:9 * D].view(step.T, 8, D)
    q.copy_(step.q)
    out = dl.attention_paged(q, dl.PagedKVCache(k, v, ks, vs), *step.seqs(cuda_device), max_q=3)
    check(step, out, None)


def test_pages_shared_by_sequences(cuda_device):
    """A common prefix: two sequences name the same pages."""
    step = Step([64, 70], [1, 2], page=32, block=8, seed=35)
    step.table[1, :2] = step.table[0, :2]
    check(step, *run(step, cuda_device))


def test_far_pages_pass_32_bits(cuda_device):
    """Page offsets beyond 2^32 bytes."""
    H, pg, D = 8, 128, 128
    pages = (1 << 32) // (H * pg * D) + 40
    codes = torch.zeros(pages, H, pg, D, dtype=torch.uint8, device=cuda_device)
    scales = torch.zeros(pages, H, 1, device=cuda_device)
    step = Step([300], [2], heads=16, kv_heads=8, page=pg, block=128, seed=36, spare_pages=0, extra_cols=0)
    far = torch.tensor([pages - 1, pages - 30, 3])
    vals = torch.zeros_like(codes)
    ks, vs = scales, scales.clone()
    for i, f in enumerate(far.tolist()):
        src = int(step.table[0, i])
        codes[f] = step.k[src].view(torch.uint8).to(cuda_device)
        vals[f] = step.v[src].view(torch.uint8).to(cuda_device)
        ks[f] = step.k_scale[src].to(cuda_device)
        vs[f] = step.v_scale[src].to(cuda_device)
    table = far.int()[None].to(cuda_device)
    _, lens, start = step.seqs(cuda_device)
    out = dl.attention_paged(step.q.to(cuda_device), dl.PagedKVCache(codes, vals, ks, vs), table, lens,
                             start, max_q=2)
    check(step, out, None)


def test_another_stream_and_a_graph(cuda_device):
    step = Step([500, 90], [1, 6], seed=37)
    first, _ = run(step, cuda_device)
    q, c, seqs = step.q.to(cuda_device), step.cache(cuda_device), step.seqs(cuda_device)
    ws = dl.Workspace(dl.attention_workspace_bytes(2, step.T, 8, 2, 128, max_q=6))
    out = torch.empty_like(first)
    side = torch.cuda.Stream(cuda_device)
    side.wait_stream(torch.cuda.current_stream(cuda_device))
    dl.attention_paged(q, c, *seqs, max_q=6, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        dl.attention_paged(q, c, *seqs, max_q=6, out=out, workspace=ws)
    seqs[1].copy_(torch.tensor([400, 90], dtype=torch.int32))   # lengths are read on the device
    graph.replay()
    torch.cuda.synchronize(cuda_device)
    step.lens[0] = 400
    check(step, out, None)


def test_workspace_serves_linears_too(cuda_device):
    """One workspace for attention and linear calls in turn: tickets return to zero."""
    step = Step([3000, 200], [1, 1], seed=38)
    n = max(dl.attention_workspace_bytes(2, 2, 8, 2, 128, max_q=1), dl.workspace_bytes(2, 1024, 1024, dl.BF16))
    ws = dl.Workspace(n)
    x = torch.randn(2, 1024, device=cuda_device).bfloat16()
    w = torch.randn(1024, 1024, device=cuda_device).bfloat16()
    y0 = dl.linear_bf16(x, w)
    a0, _ = run(step, cuda_device)
    for _ in range(3):
        a, _ = run(step, cuda_device, workspace=ws)
        y = dl.linear_bf16(x, w, workspace=ws)
        assert torch.equal(a, a0) and torch.equal(y, y0)
    assert not ws.tensor[:dl.WORKSPACE_ZERO_BYTES].any()


@pytest.mark.parametrize("group,news,withhold", [(8, 1, 1), (8, 1, 2), (8, 6, 3), (8, 8, 2)])
def test_a_withheld_tile_runs_out_and_reports(cuda_device, group, news, withhold):
    """The keys of one tile never come: the waits on it run out, the call ends with an error status
    and the context stays usable."""
    # one head, 300 tiles and more: CTA 0 has several
    step = Step([90000], [news], heads=group, kv_heads=1, page=64, block=16, seed=40)
    q, c, seqs = step.q.to(cuda_device), step.cache(cuda_device), step.seqs(cuda_device)
    first = dl.attention_paged(q, c, *seqs, max_q=news)
    torch.cuda.synchronize(cuda_device)
    assert dl.device_status() == 0
    dl.set_wait_test(20_000_000, withhold)
    try:
        dl.attention_paged(q, c, *seqs, max_q=news)
        torch.cuda.synchronize(cuda_device)
        assert dl.device_status() & 1
    finally:
        dl.set_wait_test(0, 0)
    again = dl.attention_paged(q, c, *seqs, max_q=news)
    torch.cuda.synchronize(cuda_device)
    assert dl.device_status() == 0 and torch.equal(first, again)


def test_refusals(cuda_device):
    step = Step([9], [1], seed=39)
    c, seqs, q = step.cache(cuda_device), step.seqs(cuda_device), step.q.to(cuda_device)
    with pytest.raises(ValueError, match="bfloat16"):
        dl.attention_paged(q.half(), c, *seqs, max_q=1)
    with pytest.raises(ValueError, match="tokens"):
        dl.attention_paged(q[..., :64], c, *seqs, max_q=1)
    with pytest.raises(dl.DLError, match="num_heads"):
        dl.attention_paged(q[:, :3], c, *seqs, max_q=1)
    with pytest.raises(dl.DLError, match="workspace"):
        dl.attention_paged(q, c, *seqs, max_q=1, workspace=dl.Workspace(256))
    with pytest.raises(ValueError, match="out must"):
        dl.attention_paged(q, c, *seqs, max_q=1, out=torch.empty(1, 8, 64, dtype=torch.bfloat16, device=cuda_device))
    with pytest.raises(ValueError, match="block_table"):
        dl.attention_paged(q, c, seqs[0].repeat(2, 1), *seqs[1:], max_q=1)
    with pytest.raises(dl.DLError, match="max_q"):
        dl.attention_paged(q, c, *seqs, max_q=-2)
    many = torch.zeros(1, 258, 128, dtype=torch.bfloat16, device=cuda_device)
    with pytest.raises(dl.DLError, match="q_heads"):
        dl.attention_paged(many, c, *seqs, max_q=1)
    k = torch.zeros(2, 2, 24, 128, dtype=torch.uint8, device=cuda_device)
    s = torch.zeros(2, 2, 1, device=cuda_device)
    with pytest.raises(dl.DLError, match="page_size"):
        dl.attention_paged(q, dl.PagedKVCache(k, k, s, s), *seqs, max_q=1)
    assert dl.attention_workspace_bytes(1, 1, 3, 2, 128, max_q=1) == 0
