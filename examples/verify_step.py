"""Speculative decoding with a paged 8-bit cache: the linears and the cached-attention operators
of one decode step, run together on a decoder with random weights.

A step takes, for each sequence, its last token and a few drafted ones through every layer
(linear_bf16 -> kv_append -> attention_paged -> linear_bf16 -> linear_swiglu -> linear_bf16), then
verify_draft accepts a prefix of the drafts against the target's probabilities and draws the next
token.  The drafts are drawn one by one from the decoder's own first layers.

    python examples/verify_step.py [--tokens 64] [--drafts 5] [--batch 2] [--temperature 0.3]

``--hidden 8192 --layers 80 --heads 64 --kv-heads 8 --intermediate 29568 --vocab 152064`` are the
sizes of the benchmark's decoder (about 145 GB of bf16 weights).  The linears take at most 16
tokens, so batch * (drafts + 1) <= 16.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weight_streaming_skinny_gb300 as dl  # noqa: E402


class Decoder:
    """Random weights, one paged cache a layer, and the block table that all layers share."""

    def __init__(self, *, batch, max_len, hidden=1024, layers=2, heads=8, kv_heads=2, intermediate=2816,
                 vocab=4096, page_size=64, block=16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        dim = 128 if hidden // heads >= 128 else 64

        def weight(rows, cols):
            return (torch.randn(rows, cols, device=device, generator=g) * cols ** -0.5).bfloat16()

        self.batch, self.heads, self.kv_heads, self.dim, self.device = batch, heads, kv_heads, dim, device
        self.embed = torch.randn(vocab, hidden, device=device, generator=g).bfloat16()
        self.layers = [(weight((heads + 2 * kv_heads) * dim, hidden), weight(hidden, heads * dim),
                        dl.interleave_gate_up(weight(intermediate, hidden), weight(intermediate, hidden)).contiguous(),
                        weight(hidden, intermediate)) for _ in range(layers)]
        self.head = weight(vocab, hidden)
        pages = -(-max_len // page_size)
        self.table = torch.randperm(batch * pages, generator=torch.Generator().manual_seed(seed)).int() \
            .view(batch, pages).to(device)
        self.caches = [dl.PagedKVCache.empty(batch * pages, kv_heads, dim, page_size=page_size, block=block,
                                             device=device) for _ in range(layers)]
        angle = torch.outer(torch.arange(max_len, dtype=torch.float64),
                            1e6 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim))
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)
        rows = ((heads + 2 * kv_heads) * dim, hidden, 2 * intermediate, hidden)
        cols = (hidden, heads * dim, hidden, intermediate)
        shapes = [(m, n, k, dl.BF16) for m in (1, 16) for n, k in zip(rows, cols)] + \
                 [(m, vocab, hidden, dl.BF16) for m in (1, 16)]
        attention = dl.attention_workspace_bytes(batch, 16, heads, kv_heads, dim, max_q=16)     # and of fewer tokens
        self.workspace = dl.Workspace(max(attention, *(dl.workspace_bytes(*s) for s in shapes)), device)

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def step(self, tokens, start, lens, max_new, layers=None):
        """Logits (fp32) of the new `tokens`: rows start[b] .. start[b + 1] of sequence b, which holds
        lens[b] tokens with them (all int32 tensors on the device); from the first `layers` alone if given."""
        ws = self.workspace
        x = self.embed[tokens.long()].float()
        M, H, G, D = tokens.numel(), self.heads, self.kv_heads, self.dim
        for (wqkv, wo, wgu, wdown), cache in zip(self.layers[:layers], self.caches):
            qkv = dl.linear_bf16(self.norm(x), wqkv, workspace=ws)
            q, k, v = (t.view(M, -1, D) for t in qkv.split([H * D, G * D, G * D], dim=1))
            q = dl.kv_append(q, k, v, cache, self.table, lens, start, max_q=max_new, cos=self.cos, sin=self.sin)
            a = dl.attention_paged(q, cache, self.table, lens, start, max_q=max_new, workspace=ws)
            x = x + dl.linear_bf16(a.view(M, H * D), wo, workspace=ws).float()
            h = dl.linear_swiglu(self.norm(x), wgu, workspace=ws)
            x = x + dl.linear_bf16(h, wdown, workspace=ws).float()
        logits = torch.empty(M, self.head.shape[0], device=self.device)
        dl.linear_bf16(self.norm(x), self.head, out_f32=logits, workspace=ws)
        return logits


def probabilities(logits, temperature):
    """fp32; temperature 0: all weight on the largest logit."""
    if temperature == 0:
        return torch.nn.functional.one_hot(logits.argmax(-1), logits.shape[-1]).float()
    return torch.softmax(logits / temperature, -1)


def generate(model, prompts, n, *, drafts=5, temperature=0.3, seed=0, draft_layers=1, draft_fn=None):
    """At least n new tokens for each prompt (lists of ids, equal lengths), and (accepted, offered) drafts.

    The drafts are drawn from the model's first draft_layers layers; draft_fn(history, drafts) makes
    deterministic ones instead.  The layers that draft write a draft's keys and values where the
    whole model's step then writes them again.
    """
    B, dev = len(prompts), model.device
    if B != model.batch or B * (drafts + 1) > 16:
        raise ValueError("batch * (drafts + 1) must be at most 16, the linears' token limit")
    g = torch.Generator(device=dev).manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)   # noqa: E731
    # the prompts but their last token go through in steps of 16 // B tokens
    cached, most = 0, max(1, 16 // B)
    while cached < len(prompts[0]) - 1:
        m = min(most, len(prompts[0]) - 1 - cached)
        tokens = ints([t for p in prompts for t in p[cached:cached + m]])
        cached += m
        model.step(tokens, ints([m * b for b in range(B + 1)]), ints([cached] * B), m)
    history, have = [list(p) for p in prompts], [cached] * B
    ones, wide = ints(list(range(B + 1))), ints([(drafts + 1) * b for b in range(B + 1)])
    accepted = offered = 0
    while min(len(h) - len(p) for h, p in zip(history, prompts)) < n:
        last = ints([h[-1] for h in history])
        if draft_fn is not None:
            rows, guesses = ints([draft_fn(h, drafts) for h in history]), None
        else:
            picked, guesses = [last], []
            for i in range(drafts):
                logits = model.step(picked[-1], ones, ints([c + 1 + i for c in have]), 1, layers=draft_layers)
                guesses.append(probabilities(logits, temperature))
                picked.append(torch.multinomial(guesses[-1], 1, generator=g)[:, 0].int())
            rows, guesses = torch.stack(picked[1:], 1), torch.stack(guesses, 1)
        tokens = torch.cat([last[:, None], rows], 1).view(-1)
        logits = model.step(tokens, wide, ints([c + drafts + 1 for c in have]), drafts + 1)
        target = probabilities(logits, temperature).view(B, drafts + 1, -1)
        out, count = dl.verify_draft(rows, target, torch.rand(B, drafts, device=dev, generator=g),
                                     torch.rand(B, device=dev, generator=g), draft_probs=guesses)
        out, count = out.tolist(), count.tolist()
        for b in range(B):
            # the last token and the accepted drafts stay in the cache; rejected ones are overwritten
            history[b] += out[b][:count[b] + 1]
            have[b] += count[b] + 1
        accepted += sum(count)
        offered += B * drafts
    return [h[len(p):] for h, p in zip(history, prompts)], (accepted, offered)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 64), ("drafts", 5), ("batch", 2), ("hidden", 1024), ("layers", 2), ("heads", 8),
                        ("kv-heads", 2), ("intermediate", 2816), ("vocab", 4096), ("seed", 0), ("draft-layers", 1)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--temperature", type=float, default=0.3)
    a = ap.parse_args()
    model = Decoder(batch=a.batch, max_len=64 + a.tokens + 17, hidden=a.hidden, layers=a.layers, heads=a.heads,
                    kv_heads=a.kv_heads, intermediate=a.intermediate, vocab=a.vocab, seed=a.seed)
    prompts = torch.randint(a.vocab, (a.batch, 40), generator=torch.Generator().manual_seed(a.seed)).tolist()
    texts, (accepted, offered) = generate(model, prompts, a.tokens, drafts=a.drafts, temperature=a.temperature,
                                          seed=a.seed, draft_layers=a.draft_layers)
    for t in texts:
        print(t[:a.tokens])
    print(f"{accepted} of {offered} drafted tokens accepted")


if __name__ == "__main__":
    main()
