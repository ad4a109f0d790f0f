"""norms, linears with adapters, append, attention and the pages' bookkeeping run together, as the example's
decoder uses them."""
import importlib.util
import os

import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from step_util import adapters64, assert_near, block_norm64

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "branch_step.py")
_spec = importlib.util.spec_from_file_location("branch_step_example", _PATH)
ex = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ex)


def build(rows, pages=64, **kw):
    return ex.Decoder(rows=rows, max_len=128, pages=pages, rank=8, hidden=512, layers=2, heads=4, kv_heads=2,
                      intermediate=1024, vocab=1000, page_size=16, block=4, **kw)


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def prompt(n, seed):
    return torch.randint(1000, (n,), generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("length", [16, 17, 37, 48])
def test_forks_are_copies(cuda_device, length):
    """A forked row goes on exactly as one that read the prompt itself, with other tokens after it too, and
    leaves the row that it came from alone; moving all pages to the front changes nothing."""
    shared, alone = build(4), build(4)
    p = prompt(length, length)
    first = shared.read(1, p, 2)
    for r in range(4):
        assert torch.equal(alone.read(r, p, 2), first)
    assert dl.kv_fork(shared.pool, ints([1, 1, 1]), ints([3, 0, 2])).tolist() == [1, 1, 1]
    full = length // 16
    assert int((shared.pool.refs > 0).sum()) == full + (4 if length % 16 else 0)
    assert int((alone.pool.refs > 0).sum()) == 4 * -(-length // 16)
    rows, one, start, own = ints(range(4)), ints([1] * 4), ints(range(5)), ints([2, -1, 0, 2])
    for i in range(20):
        tokens = ints([7 * i, 7 * i + 1, 300 + i, 999 - i])
        got = []
        for m in (shared, alone):
            assert dl.kv_reserve(m.pool, rows, one).tolist() == [1] * 4
            got.append(m.step(tokens, own, start, 1))
        assert torch.equal(*got), i
        if i == 5:      # give one's pages back, fork another to it, on both sides
            for m in (shared, alone):
                dl.kv_free(m.pool, ints([2]))
                assert dl.kv_fork(m.pool, ints([0]), ints([2])).tolist() == [1]
        if i == 11:
            live = int(dl.kv_compact(shared.pool))
            assert bool((shared.pool.refs[:live] > 0).all()) and not bool((shared.pool.refs[live:] > 0).any())
    for m in (shared, alone):
        dl.kv_free(m.pool, rows)
        assert not m.pool.refs.any() and not m.pool.seq_lens.any()
    assert dl.device_status() == 0


def test_a_graph_of_a_whole_step(cuda_device):
    """Reserve and step as one graph, replayed while pages fill and forks come between."""
    a, b = build(3), build(3)
    for m in (a, b):
        m.read(0, prompt(30, 1), 0)
        m.read(2, prompt(9, 2), 3)
        dl.kv_fork(m.pool, ints([0]), ints([1]))
    rows, one, start, own = ints(range(3)), ints([1] * 3), ints(range(4)), ints([0, 0, 3])
    tokens = ints([1, 2, 3])

    def step(m):
        dl.kv_reserve(m.pool, rows, one, workspace=m.workspace)
        return m.step(tokens, own, start, 1)

    assert torch.equal(step(a), step(b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a)
    for i in range(30):
        tokens.copy_(ints([i, 2 * i, 3 * i]))
        if i == 10:
            for m in (a, b):
                dl.kv_free(m.pool, ints([1]))
                dl.kv_fork(m.pool, ints([2]), ints([1]))
                dl.kv_compact(m.pool)
        graph.replay()
        assert torch.equal(out, step(b)), i
    # read, once before the graph, 30 replays; row 1 was row 2 after ten of them
    assert a.pool.seq_lens.tolist() == b.pool.seq_lens.tolist() == [30 + 31, 9 + 31, 9 + 31]
    assert torch.equal(a.pool.block_table, b.pool.block_table) and torch.equal(a.pool.refs, b.pool.refs)


def test_stages_of_a_layer(cuda_device):
    """The first layer's calls one after the other, each against its formula on what it read."""
    m = build(3)
    norm, wqkv, ad, _, _, norm2, _, _ = m.layers[0]
    h = m.embed[:16]
    own = ints([i % 6 - 1 for i in range(16)])
    _, x = dl.block_norm(None, h, pre=norm)
    y = dl.linear_bf16(x, wqkv, workspace=m.workspace)
    qkv = dl.linear_adapters(x, ad, own, y.clone(), workspace=m.workspace)
    h2, x2 = dl.block_norm(y[:, :512], h, pre=norm2)
    form = lambda n: ("rms", n.weight.cpu(), None, n.eps, n.offset)   # noqa: E731
    (_, want), (_, bound) = block_norm64(None, h.cpu(), None, form(norm), None, False, 1.0, 1.0)
    assert_near(x, want, bound, "x")
    want, bound = adapters64(x.cpu(), ad.a.cpu(), ad.b.cpu(), own.cpu(), ad.scale.cpu(), None, ad.parts, y.cpu(), False)
    assert_near(qkv, want, bound, "qkv")
    want, bound = block_norm64(y[:, :512].cpu(), h.cpu(), None, form(norm2), None, False, 1.0, 1.0)
    assert_near(h2, want[0], bound[0], "h")
    assert_near(x2, want[1], bound[1], "x")


@pytest.mark.parametrize("graph", [True, False])
def test_example_runs(cuda_device, graph):
    m = build(15, pages=15 * 3)
    prompts = [prompt(n, n) for n in (5, 16, 20)]
    texts, scores = ex.generate(m, prompts, [0, -1, 3], 20, branches=5, every=4, graph=graph)
    assert all(len(t) == 20 and all(0 <= x < 1000 for x in t) for t in texts) and all(s < 0 for s in scores)
    lens = m.pool.seq_lens.view(3, 5)
    assert lens.tolist() == [[n + 19] * 5 for n in (5, 16, 20)]
    assert dl.device_status() == 0
