"""Default workspaces and outputs of the norms, the adapters and the pages' calls belong to the stream that the
call runs on."""
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from test_call_streams_gpu import streams

pytestmark = pytest.mark.gpu


def adapters(dev, tokens, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: (torch.randn(*s, device=dev, generator=g) / 8).bfloat16()   # noqa: E731
    index = torch.arange(tokens, device=dev, dtype=torch.int32) // 70 % 3
    return rand(tokens, 256), dl.Adapters(rand(3, 16, 256), rand(3, 128, 16)), index, rand(tokens, 128)


def pool(dev):
    p = dl.PagePool.empty(dl.PagedKVCache.empty(64, 1, 64, page_size=16, block=16, device=dev), 40, 4)
    rows = torch.arange(40, device=dev, dtype=torch.int32)
    return p, rows, torch.ones_like(rows)


@pytest.mark.parametrize("tokens", [5, 40, 600])
@pytest.mark.parametrize("kind", [0, 1])
def test_default_workspace_of_adapters(cuda_device, tokens, kind):
    """A call on another stream leaves the current stream's default workspace alone."""
    args = adapters(cuda_device, tokens)
    first = dl.linear_adapters(*args)
    torch.cuda.synchronize(cuda_device)
    mine = dl._default_ws[(cuda_device.index, torch.cuda.current_stream(cuda_device).cuda_stream)]
    mine.tensor[dl.WORKSPACE_ZERO_BYTES:].fill_(0xA5)
    before = mine.tensor.clone()
    torch.cuda.synchronize(cuda_device)
    got = dl.linear_adapters(*args, stream=streams(cuda_device)[kind])
    torch.cuda.synchronize(cuda_device)
    assert torch.equal(got, first) and torch.equal(mine.tensor, before)


@pytest.mark.parametrize("kind", [0, 1])
def test_default_workspace_of_pages(cuda_device, kind):
    p, rows, ones = pool(cuda_device)
    dl.kv_reserve(p, rows, ones)
    torch.cuda.synchronize(cuda_device)
    mine = dl._default_ws[(cuda_device.index, torch.cuda.current_stream(cuda_device).cuda_stream)]
    mine.tensor[dl.WORKSPACE_ZERO_BYTES:].fill_(0xA5)
    before = mine.tensor.clone()
    torch.cuda.synchronize(cuda_device)
    done = dl.kv_reserve(p, rows, ones, stream=streams(cuda_device)[kind])
    torch.cuda.synchronize(cuda_device)
    assert bool(done.all()) and torch.equal(mine.tensor, before) and p.seq_lens.tolist() == [2] * 40


@pytest.mark.parametrize("name", ["norm", "norm of h", "adapters", "reserve", "fork", "compact"])
@pytest.mark.parametrize("kind", [0, 1])
def test_outputs(cuda_device, name, kind):
    """An output that a call on another stream makes is that stream's memory."""
    args, (p, rows, ones) = adapters(cuda_device, 40), pool(cuda_device)
    y, h = (torch.randn(40, 200, device=cuda_device) for _ in range(2))
    ws = dl.Workspace(max(dl.adapters_workspace_bytes(40, args[1]), dl.pages_workspace_bytes(p)))
    call = {"norm": lambda s: dl.block_norm(y, h, pre=dl.Norm(), stream=s),
            "norm of h": lambda s: dl.block_norm(None, h, pre=dl.Norm(), stream=s)[1:],
            "adapters": lambda s: (dl.linear_adapters(*args, workspace=ws, stream=s),),
            "reserve": lambda s: (dl.kv_reserve(p, rows, ones, workspace=ws, stream=s),),
            "fork": lambda s: (dl.kv_fork(p, rows, rows, workspace=ws, stream=s),),
            "compact": lambda s: (dl.kv_compact(p, workspace=ws, stream=s),)}[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize(cuda_device)
    got = call(streams(cuda_device)[kind])
    torch.cuda.synchronize(cuda_device)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    at, shapes = [t.data_ptr() for t in got], [(t.shape, t.dtype) for t in got]
    del got
    again = [torch.empty(s, dtype=d, device=cuda_device) for s, d in shapes for _ in range(8)]
    assert not {t.data_ptr() for t in again} & set(at)


def test_two_streams_at_once(cuda_device):
    """Calls of two streams overlap, each on its own workspace."""
    a, b = adapters(cuda_device, 2000, 1), adapters(cuda_device, 600, 2)
    want = [dl.linear_adapters(*a).clone(), dl.linear_adapters(*b).clone()]
    h = torch.randn(4000, 1024, device=cuda_device)
    r, x = dl.block_norm(h, h, pre=dl.Norm())
    torch.cuda.synchronize(cuda_device)
    side = [torch.cuda.Stream(cuda_device) for _ in range(2)]
    got = []
    for _ in range(10):
        got += [dl.linear_adapters(*a, stream=side[0]), dl.linear_adapters(*b, stream=side[1]),
                dl.block_norm(h, h, pre=dl.Norm(), stream=side[1])]
    torch.cuda.synchronize(cuda_device)
    for i in range(0, len(got), 3):
        assert torch.equal(got[i], want[0]) and torch.equal(got[i + 1], want[1])
        assert torch.equal(got[i + 2][0], r) and torch.equal(got[i + 2][1], x)
    assert dl.device_status() == 0
