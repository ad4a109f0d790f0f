"""A linear of the tensor-memory family and an attention call, launched back to back in either order."""
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import Step
from weight_streaming_skinny_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _tensor_memory_family():
    dl.set_override(dl.KERNEL_TC, 0, 0)
    yield
    dl.set_override(0, 0, 0)


@pytest.mark.parametrize("tokens", [1, 16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news", [1, 2, 4, 6, 8])
def test_back_to_back(cuda_device, tokens, dim, news):
    """The attention kernel may start, and take its tensor memory, while the linear's CTAs have not
    taken theirs."""
    L = inputs.make_layer(inputs.DTYPE_FP8_B128, tokens, 4096, 2048, bias=False, config_id=0).to(cuda_device)
    step = Step([2500, 300], [news, news], heads=16, kv_heads=2, dim=dim, page=64, seed=news)
    args = (step.q.to(cuda_device), step.cache(cuda_device), *step.seqs(cuda_device))
    y, o = dl.linear_fp8_block128(L.x, L.w, L.scales), dl.attention_paged(*args, max_q=news)
    torch.cuda.synchronize(cuda_device)
    got = []
    for _ in range(20):
        got.append((dl.linear_fp8_block128(L.x, L.w, L.scales), dl.attention_paged(*args, max_q=news)))
    torch.cuda.synchronize(cuda_device)
    assert dl.device_status() == 0
    assert all(torch.equal(a, y) and torch.equal(b, o) for a, b in got)
