"""attention_paged: a wait that runs out ends the call, however many sequences a CTA goes through.

The keys of one tile never come (nothing is in flight for them), late in a CTA that has far more
segments than it keeps descriptors of: the call has to return, report and leave the context usable.
"""
import time

import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import Step

pytestmark = pytest.mark.gpu

WAIT_NS = 20_000_000          # 20 ms
WAIT_BITS = 1 | 2             # a consumer's or the copying warp's wait, whichever runs out first


@pytest.fixture(autouse=True)
def _reset_hooks():
    dl.set_wait_test(0, 0)
    yield
    dl.set_wait_test(0, 0)


def withheld(dev, group, news, dim, length, sequences, kv_heads, withhold):
    step = Step([length], [news], heads=group * kv_heads, kv_heads=kv_heads, dim=dim, page=64, block=16, seed=withhold)
    c = step.cache(dev)
    table = step.table.expand(sequences, -1).contiguous().to(dev)
    lens = torch.full((sequences,), length, dtype=torch.int32, device=dev)
    start = torch.arange(sequences + 1, dtype=torch.int32, device=dev) * news
    q = step.q.to(dev).repeat(sequences, 1, 1)
    ws = dl.Workspace(dl.attention_workspace_bytes(sequences, sequences * news, group * kv_heads, kv_heads, dim, max_q=news))
    call = lambda: dl.attention_paged(q, c, table, lens, start, max_q=news, workspace=ws)   # noqa: E731
    first = call()
    torch.cuda.synchronize(dev)
    assert dl.device_status() == 0
    dl.set_wait_test(WAIT_NS, withhold)
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize(dev)
    elapsed = time.perf_counter() - t0
    dl.set_wait_test(0, 0)
    flags = dl.device_status()
    assert flags & WAIT_BITS, f"error word 0x{flags:x}: the wait did not run out"
    assert elapsed < 5.0, f"the call took {elapsed:.2f} s with a 20 ms wait limit"
    again = call()
    torch.cuda.synchronize(dev)
    assert dl.device_status() == 0 and torch.equal(first, again)


@pytest.mark.parametrize("group,news", [(8, 1), (8, 2), (8, 4), (8, 6), (8, 8)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("withhold", [1, 2, 10, 11, 12, 15])
def test_many_segments_of_a_cta(cuda_device, group, news, dim, withhold):
    """1000 sequences of one tile each, 8 heads: at least 17 segments on each of at most 456 CTAs."""
    withheld(cuda_device, group, news, dim, 90, 1000, 8, withhold)


@pytest.mark.parametrize("group,news", [(8, 1), (8, 6)])
@pytest.mark.parametrize("withhold", [23, 24])
def test_segments_of_two_tiles(cuda_device, group, news, withhold):
    """The first and the second tile of a segment past the tenth."""
    withheld(cuda_device, group, news, 128, 200, 1000, 8, withhold)
