"""What a captured call reads of a PagePool outlives the object, with the caches."""
import gc
import weakref

import pytest
import torch

import weight_streaming_skinny_gb300 as dl

pytestmark = pytest.mark.gpu


def make(dev, layers=3):
    caches = [dl.PagedKVCache.empty(24, 2, 64, page_size=16, block=16, device=dev) for _ in range(layers)]
    g = torch.Generator(device=dev).manual_seed(1)
    for c in caches:
        for t in (c.k, c.v):
            t.copy_(torch.randint(0, 256, t.shape, device=dev, generator=g))
        for t in (c.k_scale, c.v_scale):
            t.copy_(torch.rand(t.shape, device=dev, generator=g))
    return caches


def buffers(pool):
    """Weak references to the device buffers that a pool has made for itself."""
    own = {id(t) for t in (pool.refs, pool.block_table, pool.seq_lens)}
    return [weakref.ref(t) for t in vars(pool).values() if isinstance(t, torch.Tensor) and id(t) not in own]


def test_descriptions_belong_to_the_caches(cuda_device):
    caches = make(cuda_device)
    pool = dl.PagePool.empty(caches, 4, 4)
    held = buffers(pool)
    assert held
    del pool
    gc.collect()
    assert all(r() is not None for r in held)
    again = dl.PagePool.empty(caches, 5, 4)          # the same caches: nothing more is held
    assert len(buffers(again)) == len(held) and all(a() is b() for a, b in zip(buffers(again), held))
    del again, caches
    gc.collect()
    assert all(r() is None for r in held)


def test_a_graph_without_its_pool(cuda_device):
    """Captured fork and compact, replayed after the pool is gone and its place could have been taken."""
    caches, same = make(cuda_device), make(cuda_device)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=cuda_device)   # noqa: E731
    pool, other = dl.PagePool.empty(caches, 4, 4), dl.PagePool.empty(same, 4, 4)
    for p in (pool, other):
        dl.kv_reserve(p, ints(0, 1), ints(20, 37))
        dl.kv_free(p, ints(0))
    ws, parents, children = dl.Workspace(dl.pages_workspace_bytes(pool)), ints(1, 1), ints(0, 3)
    torch.cuda.synchronize(cuda_device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        done = dl.kv_fork(pool, parents, children, workspace=ws)
        live = dl.kv_compact(pool, workspace=ws)
    state = pool.refs, pool.block_table, pool.seq_lens
    del pool
    gc.collect()
    filled = [torch.full((n,), 0xA5, dtype=torch.uint8, device=cuda_device) for n in (88, 264, 512, 1024) for _ in range(300)]
    torch.cuda.synchronize(cuda_device)
    graph.replay()
    want = dl.kv_fork(other, parents, children), dl.kv_compact(other)
    torch.cuda.synchronize(cuda_device)
    assert torch.equal(done, want[0]) and torch.equal(live, want[1])
    for a, b in zip(state, (other.refs, other.block_table, other.seq_lens)):
        assert torch.equal(a, b)
    for c, d in zip(caches, same):
        for n in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(getattr(c, n), getattr(d, n))
    assert all(bool((t == 0xA5).all()) for t in filled)
