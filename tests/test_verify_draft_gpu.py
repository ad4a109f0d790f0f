"""verify_draft against whole numbers in Python: equal tokens and counts."""
import numpy as np
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import reference_verify

pytestmark = pytest.mark.gpu


def make(B, S, V, seed, kind=torch.float32, close=0.5, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(B, S + 1, V, generator=g)
    target = torch.softmax(logits, -1).to(kind)
    guess = torch.softmax(logits[:, :S] + close * torch.randn(B, S, V, generator=g), -1).to(kind)
    drafts = torch.multinomial(guess.float().reshape(-1, V), 1, generator=g).view(B, S).int() if S else \
        torch.zeros(B, 0, dtype=torch.int32)
    return drafts, target, guess, torch.rand(B, S, generator=g), torch.rand(B, generator=g)


def check(dev, drafts, target, guess, u, u_next, lens=None):
    on = lambda x: None if x is None else x.to(dev).contiguous()   # noqa: E731
    tokens, count = dl.verify_draft(on(drafts), on(target), on(u), on(u_next), draft_probs=on(guess),
                                    draft_lens=on(lens))
    f = lambda x: None if x is None else x.float().numpy()   # noqa: E731
    want = reference_verify(drafts.numpy(), f(target), f(guess), f(u), f(u_next),
                            None if lens is None else lens.numpy())
    assert np.array_equal(count.cpu().numpy(), want[1])
    assert np.array_equal(tokens.cpu().numpy(), want[0])
    return want


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (3, 2, 2), (5, 4, 31), (4, 5, 1000), (3, 7, 4099), (2, 15, 32768),
                                   (2, 3, 152064), (1, 5, 152063), (70, 1, 257), (6, 0, 999)])
def test_matches_whole_numbers(cuda_device, kind, with_draft, B, S, V):
    drafts, target, guess, u, u_next = make(B, S, V, B * 100 + S + V, kind)
    check(cuda_device, drafts, target, guess if with_draft and S else None, u, u_next)


def test_all_counts_occur(cuda_device):
    drafts, target, guess, u, u_next = make(64, 5, 500, 1, close=0.6)
    count = check(cuda_device, drafts, target, guess, u, u_next)[1]
    assert set(count.tolist()) == set(range(6))


def test_largest_vocabulary_and_ones(cuda_device):
    """Every probability 1 in 262144 entries: the sum is 2^62."""
    V = 1 << 18
    target = torch.ones(2, 1, V)
    drafts, u = torch.zeros(2, 0, dtype=torch.int32), torch.zeros(2, 0)
    want = check(cuda_device, drafts, target, None, u, torch.tensor([0.0, 0.99999994]))[0]
    assert want[:, 0].tolist() == [0, V - 1]


def test_random_numbers_at_their_ends(cuda_device):
    drafts, target, guess, u, _ = make(4, 3, 700, 3)
    u = torch.tensor([[0.0] * 3, [0.99999994] * 3, [0.5] * 3, [0.0] * 3])
    check(cuda_device, drafts, target, guess, u, torch.tensor([0.0, 0.99999994, 2.0 ** -24, 0.5]))


def test_ragged_drafts(cuda_device):
    drafts, target, guess, u, u_next = make(7, 6, 321, 4)
    lens = torch.tensor([0, 1, 2, 3, 4, 5, 6], dtype=torch.int32)
    drafts[2, 2:] = -7                      # past a sequence's end: not read
    check(cuda_device, drafts, target, guess, u, u_next, lens)
    check(cuda_device, drafts, target, None, u, u_next, lens)


def test_equal_distributions_accept_all(cuda_device):
    drafts, target, _, u, u_next = make(8, 4, 600, 5)
    check(cuda_device, drafts, target, target[:, :4], u, u_next)


def test_nothing_left_falls_back(cuda_device):
    """A rejected token whose residual is zero everywhere draws from the target; an empty row has no token."""
    drafts = torch.tensor([[3], [3], [9], [2]], dtype=torch.int32)
    target = torch.zeros(4, 2, 50)
    target[0, 0, 7] = 0.5
    target[2, 0, 4] = 1.0
    guess = torch.zeros(4, 1, 50)
    guess[0, 0, 7] = 0.75
    guess[2, 0, 9] = 1.0
    target[3, 0] = 0.02
    guess[3, 0] = 0.02
    u = torch.tensor([[0.5]] * 3 + [[1.0]])
    want = check(cuda_device, drafts, target, guess, u, torch.full((4,), 0.3))
    assert want[0][:, 0].tolist() == [7, -1, 4, 15]


def test_tokens_out_of_range_and_nan(cuda_device):
    drafts, target, guess, u, u_next = make(5, 3, 400, 6)
    u.zero_()
    drafts[0, 0], drafts[1, 1], drafts[2, 2] = -1, 400, 2 ** 31 - 1
    target[3, 1, int(drafts[3, 1])] = float("nan")
    guess[4, 0, int(drafts[4, 0])] = float("nan")
    target[4, 0, 17] = float("nan")
    want = check(cuda_device, drafts, target, guess, u, u_next)
    assert want[1].tolist() == [0, 1, 2, 1, 0]
    check(cuda_device, drafts, target, None, u, u_next)


def test_ties_and_zero_probabilities(cuda_device):
    """Zeros before and after the drawn token are never drawn."""
    target = torch.zeros(16, 1, 3000)
    target[:, 0, 1000:1004] = 0.25
    u_next = torch.arange(16) / 16.0
    want = check(cuda_device, torch.zeros(16, 0, dtype=torch.int32), target, None, torch.zeros(16, 0), u_next)
    assert want[0][:, 0].tolist() == [1000 + i // 4 for i in range(16)]


def test_frequencies_follow_the_target(cuda_device):
    """The accepted-or-drawn first token is distributed as the target, whatever the draft's
    distribution: 20000 trials over 8 tokens, each count within 5 standard deviations."""
    n, g = 20000, torch.Generator().manual_seed(8)
    p = torch.tensor([0.3, 0.2, 0.15, 0.1, 0.1, 0.05, 0.05, 0.05])
    d = torch.tensor([0.05, 0.05, 0.3, 0.2, 0.1, 0.1, 0.1, 0.1])
    drafts = torch.multinomial(d, n, True, generator=g).int()[:, None].contiguous()
    target = p.repeat(n, 2, 1).to(cuda_device)
    guess = d.repeat(n, 1, 1).to(cuda_device)
    u, un = torch.rand(n, 1, generator=g), torch.rand(n, generator=g)
    tokens, _ = dl.verify_draft(drafts.to(cuda_device), target, u.to(cuda_device), un.to(cuda_device),
                                draft_probs=guess)
    got = torch.bincount(tokens[:, 0].long().cpu(), minlength=8) / n
    assert ((got - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all()


def test_repeats_and_another_stream(cuda_device):
    args = [x.to(cuda_device) for x in make(9, 4, 5000, 9)]
    first = dl.verify_draft(args[0], args[1], args[3], args[4], draft_probs=args[2])
    side = torch.cuda.Stream(cuda_device)
    side.wait_stream(torch.cuda.current_stream(cuda_device))
    for _ in range(3):
        again = dl.verify_draft(args[0], args[1], args[3], args[4], draft_probs=args[2], stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_refusals(cuda_device):
    drafts, target, guess, u, u_next = (x.to(cuda_device) for x in make(2, 3, 40, 10))
    with pytest.raises(ValueError, match="int32"):
        dl.verify_draft(drafts.long(), target, u, u_next)
    with pytest.raises(ValueError, match="target_probs"):
        dl.verify_draft(drafts, target[:, :3].contiguous(), u, u_next)
    with pytest.raises(ValueError, match="float32 or"):
        dl.verify_draft(drafts, target.half(), u, u_next)
    with pytest.raises(ValueError, match="draft_probs"):
        dl.verify_draft(drafts, target, u, u_next, draft_probs=guess.bfloat16())
    with pytest.raises(ValueError, match="CUDA"):
        dl.verify_draft(drafts.cpu(), target.cpu(), u.cpu(), u_next.cpu())
    with pytest.raises(ValueError, match="u_accept"):
        dl.verify_draft(drafts, target, u[:, :1].contiguous(), u_next)
    with pytest.raises(dl.DLError, match="vocab"):
        z = torch.zeros(1, 1, (1 << 18) + 1, device=cuda_device)
        dl.verify_draft(drafts[:1, :0].contiguous(), z, u[:1, :0].contiguous(), u_next[:1].contiguous())
    with pytest.raises(dl.DLError, match="drafts"):
        z = torch.zeros(1, 65, 4, device=cuda_device)
        dl.verify_draft(torch.zeros(1, 64, dtype=torch.int32, device=cuda_device), z,
                        torch.zeros(1, 64, device=cuda_device), u_next[:1].contiguous())
