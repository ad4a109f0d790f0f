"""Default buffers of the cached-attention calls belong to the stream that the call runs on."""
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import Step, rope_tables

pytestmark = pytest.mark.gpu


def streams(dev):
    side = torch.cuda.Stream(dev)
    return [side, side.cuda_stream]               # as an object, and as a number


@pytest.mark.parametrize("kind", [0, 1])
def test_default_workspace(cuda_device, kind):
    """A call on another stream leaves the current stream's default workspace alone."""
    step = Step([5003], [2], heads=8, kv_heads=1, page=64, seed=1)
    q, c, seqs = step.q.to(cuda_device), step.cache(cuda_device), step.seqs(cuda_device)
    first = dl.attention_paged(q, c, *seqs, max_q=2)
    torch.cuda.synchronize(cuda_device)
    mine = dl._default_ws[(cuda_device.index, torch.cuda.current_stream(cuda_device).cuda_stream)]
    mine.tensor[dl.WORKSPACE_ZERO_BYTES:].fill_(0xA5)
    before = mine.tensor.clone()
    torch.cuda.synchronize(cuda_device)
    got = dl.attention_paged(q, c, *seqs, max_q=2, stream=streams(cuda_device)[kind])
    torch.cuda.synchronize(cuda_device)
    assert torch.equal(got, first) and torch.equal(mine.tensor, before)


def test_linear_default_workspace(cuda_device):
    """The linears take theirs from the same place."""
    x = torch.randn(2, 8192, device=cuda_device).bfloat16()
    w = torch.randn(1024, 8192, device=cuda_device).bfloat16()
    first = dl.linear_bf16(x, w)
    torch.cuda.synchronize(cuda_device)
    mine = dl._default_ws[(cuda_device.index, torch.cuda.current_stream(cuda_device).cuda_stream)]
    mine.tensor[dl.WORKSPACE_ZERO_BYTES:].fill_(0xA5)
    before = mine.tensor.clone()
    torch.cuda.synchronize(cuda_device)
    got = dl.linear_bf16(x, w, stream=streams(cuda_device)[0])
    torch.cuda.synchronize(cuda_device)
    assert torch.equal(got, first) and torch.equal(mine.tensor, before)


def test_an_outgrown_workspace_stays(cuda_device):
    """A larger call takes a larger buffer; the one that earlier calls or a graph name is not freed."""
    side = torch.cuda.Stream(cuda_device)
    small = Step([900], [1], heads=8, kv_heads=1, page=64, seed=2)
    args = (small.q.to(cuda_device), small.cache(cuda_device), *small.seqs(cuda_device))
    torch.cuda.synchronize(cuda_device)
    with torch.cuda.stream(side):
        want = dl.attention_paged(*args, max_q=1)
        side.synchronize()
        at = dl._default_ws[(cuda_device.index, side.cuda_stream)].addr
        out = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            dl.attention_paged(*args, max_q=1, out=out)
        big = Step([900], [8], heads=8, kv_heads=1, page=64, seed=3)
        dl.attention_paged(big.q.to(cuda_device), big.cache(cuda_device), *big.seqs(cuda_device), max_q=8)
        side.synchronize()
        now = dl._default_ws[(cuda_device.index, side.cuda_stream)]
        assert now.addr != at
        held = [torch.empty(n, dtype=torch.uint8, device=cuda_device) for n in (now.nbytes // 8, now.nbytes // 2, now.nbytes)]
        assert not any(t.data_ptr() <= at < t.data_ptr() + t.numel() for t in held)
        graph.replay()
        side.synchronize()
    assert torch.equal(out, want)


def calls(dev):
    step = Step([70, 40], [3, 2], seed=4)
    cos, sin = (torch.from_numpy(t).to(dev) for t in rope_tables(80, 128))
    q, k, v = (t.to(dev) for t in (step.q, step.new_k, step.new_v))
    c, seqs = step.cache(dev), step.seqs(dev)
    ws = dl.Workspace(dl.attention_workspace_bytes(2, 5, 8, 2, 128, max_q=3))
    drafts = torch.zeros(40, 3, dtype=torch.int32, device=dev)
    target = torch.full((40, 4, 64), 1 / 64, device=dev)
    u, un = torch.rand(40, 3, device=dev), torch.rand(40, device=dev)
    return {"attention": lambda s: (dl.attention_paged(q, c, *seqs, max_q=3, workspace=ws, stream=s),),
            "append": lambda s: (dl.kv_append(q, k, v, c, *seqs, max_q=3, cos=cos, sin=sin, stream=s),),
            "verify": lambda s: dl.verify_draft(drafts, target, u, un, stream=s)}


@pytest.mark.parametrize("name", ["attention", "append", "verify"])
@pytest.mark.parametrize("kind", [0, 1])
def test_outputs(cuda_device, name, kind):
    """An output that a call on another stream makes is that stream's memory: what the current stream
    frees is not written while it may still use it, nor given away while the call may still write it."""
    call = calls(cuda_device)[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize(cuda_device)
    got = call(streams(cuda_device)[kind])
    torch.cuda.synchronize(cuda_device)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    at = [t.data_ptr() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    again = [torch.empty(s, dtype=d, device=cuda_device) for s, d in shapes for _ in range(8)]
    assert not {t.data_ptr() for t in again} & set(at)
