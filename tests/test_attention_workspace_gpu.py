"""attention_paged's workspace: its size is a bound for every smaller step."""
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 6, 7, 8, 12, 16, 64, 96, 128])
def test_a_larger_bound_is_never_smaller(cuda_device, dim, group):
    last = 0
    for max_q in list(range(1, 17)) + [24, 33, 64, 65, 100, 4096]:
        n = dl.attention_workspace_bytes(1, max_q, group, 1, dim, max_q=max_q)
        assert n >= last, max_q
        last = n
        # the tokens of all sequences bound a sequence's, and the batch does not matter
        assert dl.attention_workspace_bytes(9, 9 * max_q, 2 * group, 2, dim, max_q=max_q) == n
        assert dl.attention_workspace_bytes(1, max_q, group, 1, dim, max_q=2 * max_q) == n


@pytest.mark.parametrize("dim,most,news", [(128, 12, range(1, 13)), (64, 5, range(1, 6))])
def test_one_workspace_serves_every_smaller_step(cuda_device, dim, most, news):
    ws = dl.Workspace(dl.attention_workspace_bytes(1, most, 8, 1, dim, max_q=most))
    for n in news:
        step = Step([700], [n], heads=8, kv_heads=1, dim=dim, page=64, seed=n)
        args = (step.q.to(cuda_device), step.cache(cuda_device), *step.seqs(cuda_device))
        a = dl.attention_paged(*args, max_q=n, workspace=ws)
        assert torch.equal(a, dl.attention_paged(*args, max_q=n))


def test_a_workspace_of_another_device_is_refused(cuda_device):
    """Its address would mean nothing on the cache's device."""
    step = Step([40], [1], seed=9)
    ws = object.__new__(dl.Workspace)
    ws.tensor = torch.zeros(1 << 24, dtype=torch.uint8)
    ws.nbytes, ws.addr = ws.tensor.numel(), ws.tensor.data_ptr()
    with pytest.raises(ValueError, match="workspace is on cpu"):
        dl.attention_paged(step.q.to(cuda_device), step.cache(cuda_device), *step.seqs(cuda_device), max_q=1, workspace=ws)
