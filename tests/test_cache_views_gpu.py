"""PagedKVCache of views whose one head or one page has a stride that says nothing."""
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import Step

pytestmark = pytest.mark.gpu


def both(dev, step, make):
    """The operators on a dense cache and on views with the same content: equal results."""
    results = []
    for view in (False, True):
        c = step.cache(dev)
        if view:
            c = dl.PagedKVCache(*(make(t) for t in (c.k, c.v, c.k_scale, c.v_scale)))
        q, k, v = (t.to(dev) for t in (step.q, step.new_k, step.new_v))
        q = dl.kv_append(q, k, v, c, *step.seqs(dev), max_q=step.max_q)
        out = dl.attention_paged(q, c, *step.seqs(dev), max_q=step.max_q)
        torch.cuda.synchronize(dev)
        results.append([q, out, c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone(), c.k_scale.clone(), c.v_scale.clone()])
    assert dl.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_one_head_of_a_token_major_layout(cuda_device):
    """[pages, tokens, heads, dim] seen as [pages, heads, tokens, dim]: with one head its stride is one token's."""
    step = Step([150, 33], [3, 2], heads=4, kv_heads=1, page=32, block=8, seed=1)

    def make(t):
        by_token = torch.empty(t.transpose(1, 2).shape, dtype=t.dtype, device=t.device)
        by_token.copy_(t.transpose(1, 2))
        t = by_token.transpose(1, 2)
        assert t.stride(1) == (t.shape[3] if t.dim() == 4 else 1)
        return t
    both(cuda_device, step, make)


@pytest.mark.parametrize("heads", [1, 2])
def test_one_page(cuda_device, heads):
    """A page that is a slice of others, for the keys and not for the values."""
    step = Step([30], [3], heads=2 * heads, kv_heads=heads, page=32, block=8, spare_pages=0, seed=2)
    count = [0]

    def make(t):
        count[0] += 1
        if count[0] % 2:
            return torch.cat([t] * 3).transpose(0, 1).contiguous().transpose(0, 1)[:1]
        return t.as_strided(t.shape, (1,) + t.stride()[1:])
    if heads == 2:
        make = lambda t: t.as_strided(t.shape, (1,) + t.stride()[1:])   # noqa: E731
    both(cuda_device, step, make)
