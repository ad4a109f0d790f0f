"""The example's decode loop: drafted and one-by-one decoding agree, and a step's layer matches a
plain 64-bit evaluation of what it read."""
import importlib.util
import os

import pytest
import torch

import weight_streaming_skinny_gb300 as dl

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
_spec = importlib.util.spec_from_file_location("verify_step_example", _PATH)
ex = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ex)


def build(batch, **kw):
    return ex.Decoder(batch=batch, max_len=160, hidden=512, layers=2, heads=4, kv_heads=2, intermediate=1024,
                      vocab=1000, page_size=16, block=4, **kw)


def one_by_one(tokens, more=0):
    """Decoding a token a step: after each token the largest logit's id and its margin over the next
    one in units of the logits' spread; `more` tokens beyond the given ones are its own."""
    m = build(1)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    h, best, margins = list(tokens), [], []
    for i in range(len(tokens) + more):
        logits = m.step(ints([h[i]]), ints([0, 1]), ints([i + 1]), 1)[0]
        top = logits.topk(2)
        margins.append(float((top.values[0] - top.values[1]) / logits.std()))
        best.append(int(top.indices[0]))
        if i + 1 >= len(h):
            h.append(best[-1])
    return best, margins, h


def test_drafted_decoding_equals_one_by_one(cuda_device):
    """At temperature 0 every token is the largest logit's, whatever the drafts were.  Keys and values
    are rounded to 8 bits (relative 2^-4 at most) under scales that rejected drafts may have
    grown, so a near tie may fall the other way: tokens count where the margin is a tenth of the
    logits' spread or more."""
    prompts = torch.randint(1000, (2, 21), generator=torch.Generator().manual_seed(1)).tolist()
    got, _ = ex.generate(build(2), prompts, 40, drafts=5, temperature=0)
    clear = 0
    for p, t in zip(prompts, got):
        best, margins, _ = one_by_one(p + t)
        for i, token in enumerate(t):
            if margins[len(p) - 1 + i] >= 0.1:
                assert token == best[len(p) - 1 + i], i
                clear += 1
    assert clear >= 20


def test_right_drafts_are_accepted(cuda_device):
    """Drafts made by the same decoder one by one: all accepted but for near ties."""
    prompts = torch.randint(1000, (2, 11), generator=torch.Generator().manual_seed(3)).tolist()

    def oracle(history, drafts):
        return one_by_one(history, drafts - 1)[2][len(history):]

    _, (accepted, offered) = ex.generate(build(2), prompts, 24, drafts=5, temperature=0, draft_fn=oracle)
    assert accepted >= 0.8 * offered


def test_sampling_runs_and_counts(cuda_device):
    prompts = torch.randint(1000, (4, 9), generator=torch.Generator().manual_seed(2)).tolist()
    texts, (accepted, offered) = ex.generate(build(4), prompts, 12, drafts=3, temperature=0.7)
    assert all(len(t) >= 12 and all(0 <= x < 1000 for x in t) for t in texts)
    assert 0 <= accepted <= offered
    assert dl.device_status() == 0


def test_a_step_in_a_graph(cuda_device):
    """One step of drafts captured and replayed with other tokens and lengths."""
    m = build(2)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    start, lens, tokens = ints([0, 4, 8]), ints([4, 4]), ints(list(range(8)))
    for _ in range(2):
        m.step(tokens, start, lens, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = m.step(tokens, start, lens, 4)
    lens.copy_(ints([8, 8]))
    tokens.copy_(ints([9, 8, 7, 6, 5, 4, 3, 2]))
    graph.replay()
    got = logits.clone()
    again = m.step(tokens, start, lens, 4)
    assert torch.equal(got, again)
