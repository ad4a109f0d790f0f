"""Lists of the pages' calls and done in the same memory: lists are read before done is written."""
import pytest
import torch

import weight_streaming_skinny_gb300 as dl

pytestmark = pytest.mark.gpu


def pool(dev, rows=2100):
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)   # noqa: E731
    return dl.PagePool([], zeros(rows, 4) - 1, zeros(rows), zeros(4 * rows), page_size=8)


@pytest.mark.parametrize("n", [5, 2048])
@pytest.mark.parametrize("where", ["tokens", "rows", "behind tokens", "before tokens"])
def test_reserve(cuda_device, n, where):
    rows = torch.randperm(n, generator=torch.Generator().manual_seed(n)).int().to(cuda_device)
    tokens = torch.arange(n, dtype=torch.int32, device=cuda_device) % 33 - 1
    want, p = pool(cuda_device), pool(cuda_device)
    done = dl.kv_reserve(want, rows, tokens).clone()
    assert int(done.sum()) < n and bool(done.any())
    wide = torch.zeros(n + 2, dtype=torch.int32, device=cuda_device)
    wide[1:-1] = rows if where == "rows" else tokens
    lists = {"rows": (wide[1:-1], tokens, wide[1:-1])}.get(
        where, (rows, wide[1:-1], {"tokens": wide[1:-1], "behind tokens": wide[2:], "before tokens": wide[:-2]}.get(where)))
    got = dl.kv_reserve(p, lists[0], lists[1], out_done=lists[2])
    assert torch.equal(got, done)
    for name in ("refs", "block_table", "seq_lens"):
        assert torch.equal(getattr(p, name), getattr(want, name))


@pytest.mark.parametrize("n", [5, 1024])
@pytest.mark.parametrize("where", ["parents", "children"])
def test_fork(cuda_device, n, where):
    first = torch.arange(n, dtype=torch.int32, device=cuda_device)
    want, p = pool(cuda_device), pool(cuda_device)
    for x in (want, p):
        dl.kv_reserve(x, first, first % 30)
    parents, children = first.flip(0).contiguous(), first + n
    children[2] = 1                      # refused: not empty
    done = dl.kv_fork(want, parents, children).clone()
    assert int(done.sum()) == n - 1
    lists = {"parents": parents.clone(), "children": children.clone()}
    got = dl.kv_fork(p, *lists.values(), out_done=lists[where])
    assert torch.equal(got, done)
    for name in ("refs", "block_table", "seq_lens"):
        assert torch.equal(getattr(p, name), getattr(want, name))
