"""verify_draft at vocabularies around every whole number of entries of a warp's run."""
import numpy as np
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import reference_verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups", range(1, 9))
@pytest.mark.parametrize("more", [-129, -1, 0, 1, 4, 133])
def test_runs_of_one_to_eight_groups(cuda_device, kind, groups, more):
    """16 CTAs of 16 warps take 32768 entries as one group of 128 a warp, 262144 as eight; the
    drawn token lies anywhere, in the last entries too."""
    V = min(32768 * groups + more, 262144)
    B, S = 3, 1
    g = torch.Generator().manual_seed(groups * 1000 + more)
    target = torch.softmax(2 * torch.randn(B, S + 1, V, generator=g), -1).to(kind)
    guess = torch.softmax(2 * torch.randn(B, S, V, generator=g), -1).to(kind)
    drafts = torch.randint(0, V, (B, S), generator=g, dtype=torch.int32)
    u, u_next = torch.rand(B, S, generator=g), torch.tensor([0.0, 0.37, 1 - 2.0 ** -24])
    tokens, count = dl.verify_draft(*(t.to(cuda_device) for t in (drafts, target, u, u_next)),
                                    draft_probs=guess.to(cuda_device))
    torch.cuda.synchronize(cuda_device)
    want, want_count = reference_verify(drafts.numpy(), target.float().numpy(), guess.float().numpy(), u.numpy(),
                                        u_next.numpy())
    assert np.array_equal(tokens.cpu().numpy(), want) and np.array_equal(count.cpu().numpy(), want_count)
