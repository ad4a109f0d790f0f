"""A thread's first call of CUDA may be one of the library's: every entry point that describes tensors to the copy
engine, with all buffers made by another thread.
"""
import threading

import pytest
import torch

import weight_streaming_skinny_gb300 as dl

pytestmark = pytest.mark.gpu


def calls(dev):
    g = torch.Generator(device=dev).manual_seed(1)
    rand = lambda *s: (torch.randn(*s, device=dev, generator=g) / 8).bfloat16()   # noqa: E731
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)   # noqa: E731
    x, w, out = rand(4, 512), rand(256, 512), torch.empty(4, 256, dtype=torch.bfloat16, device=dev)
    codes = torch.randint(0, 100, (256, 512), dtype=torch.uint8, device=dev, generator=g)
    scales = torch.ones(2, 4, device=dev)
    ws = dl.Workspace(64 << 20, dev)
    yield "linear_bf16", lambda: dl.linear_bf16(x, w, out=out, workspace=ws)
    yield "linear_fp8", lambda: dl.linear_fp8_block128(x, codes, scales, out=out, workspace=ws)
    cache = dl.PagedKVCache.empty(4, 2, 64, device=dev)
    cache.k.copy_(torch.randint(0, 100, cache.k.shape, device=dev, generator=g))
    cache.v.copy_(torch.randint(0, 100, cache.v.shape, device=dev, generator=g))
    cache.k_scale.fill_(0.01)
    cache.v_scale.fill_(0.02)
    q, seen = rand(2, 4, 64), torch.empty(2, 4, 64, dtype=torch.bfloat16, device=dev)
    table, lens, start = ints(0, 1, 2, 3)[None], ints(200), ints(0, 2)
    yield "attention_paged", lambda: dl.attention_paged(q, cache, table, lens, start, max_q=2, out=seen, workspace=ws)
    ad, many = dl.Adapters(rand(2, 16, 512), rand(2, 128, 16)), rand(300, 512)
    index, base = torch.arange(300, device=dev, dtype=torch.int32) // 150, rand(300, 128)
    got = torch.empty_like(base)
    yield "linear_adapters", lambda: dl.linear_adapters(many, ad, index, base, out=got, workspace=ws)


@pytest.mark.parametrize("name", ["linear_bf16", "linear_fp8", "attention_paged", "linear_adapters"])
def test_a_new_thread(cuda_device, name):
    call = dict(calls(cuda_device))[name]
    want = call().clone()
    torch.cuda.synchronize(cuda_device)
    got = []

    def run():
        try:
            got.append(call())
        except Exception as e:           # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize(cuda_device)
    assert isinstance(got[0], torch.Tensor), got[0]
    assert torch.equal(got[0], want)
