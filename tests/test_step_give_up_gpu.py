"""block_norm and linear_adapters: a wait that runs out ends the call.

One stage of CTA 0 never comes (nothing is in flight for it): the call has to return, report and leave the
context usable; the next one gives what the first did.
"""
import time

import pytest
import torch

import weight_streaming_skinny_gb300 as dl

pytestmark = pytest.mark.gpu

WAIT_NS = 20_000_000          # 20 ms
WAIT_BITS = 1 | 2             # a consumer's or a copying thread's wait, whichever runs out first


@pytest.fixture(autouse=True)
def _reset_hooks():
    dl.set_wait_test(0, 0)
    yield
    dl.set_wait_test(0, 0)


def withheld(dev, call, withhold):
    first = [t.clone() for t in call()]
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
    assert dl.device_status() == 0 and all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dim", [2048, 8192])
@pytest.mark.parametrize("withhold", [1, 2, 4])
def test_norm(cuda_device, dim, withhold):
    """3000 rows, at least 4 to a CTA."""
    g = torch.Generator(device=cuda_device).manual_seed(dim)
    y, h = (torch.randn(3000, dim, device=cuda_device, generator=g) for _ in range(2))
    y = y.bfloat16()
    withheld(cuda_device, lambda: dl.block_norm(y, h, pre=dl.Norm()), withhold)


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("withhold", [1, 3, 5])
def test_adapters(cuda_device, mixed, f32, withhold):
    """2000 tokens of two adapters: 16 tiles, 5 stages to a CTA of a first product and more blocks to one of a second."""
    g = torch.Generator(device=cuda_device).manual_seed(3)
    rand = lambda *s: (torch.randn(*s, device=cuda_device, generator=g) / 8).bfloat16()   # noqa: E731
    ad = dl.Adapters(rand(2, 32, 4096), rand(2, 20480, 32))
    index = torch.arange(2000, device=cuda_device, dtype=torch.int32)
    index = index % 2 if mixed else index // 1000
    x, base = rand(2000, 4096), rand(2000, 20480)
    out32 = torch.empty(2000, 20480, device=cuda_device) if f32 else None
    ws = dl.Workspace(dl.adapters_workspace_bytes(2000, ad))

    def call():
        out = dl.linear_adapters(x, ad, index, base, out_f32=out32, workspace=ws)
        return (out, out32.clone()) if f32 else (out,)

    withheld(cuda_device, call, withhold)
