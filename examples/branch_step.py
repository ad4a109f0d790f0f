"""Several continuations of each user's prompt over one pool of cache pages, every user with an
adapter of their own: norms, adapters and page bookkeeping around the linears and the attention of a
decode step, on a decoder with random weights.

A step takes the new token of every continuation through all layers (block_norm -> linear_bf16 +
linear_adapters -> kv_append -> attention_paged -> linear_bf16 + linear_adapters -> block_norm ->
linear_swiglu -> linear_bf16).  A prompt is read once, into one row; kv_fork makes the other rows, which
share its full pages.  Every few tokens a user's continuations are taken up from the likeliest
one: kv_free gives the others' pages back and kv_fork copies it to their rows.  Lengths, tables and page
counts stay on the device, so a step with its kv_reserve replays as one graph.

    python examples/branch_step.py [--users 3] [--branches 5] [--tokens 48] [--every 8]

The linears take at most 16 tokens, so users * branches <= 16.
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
    """Random weights and adapters, one paged cache a layer, and the pool of their pages with `rows` rows."""

    def __init__(self, *, rows, max_len, pages, adapters=4, rank=16, hidden=1024, layers=2, heads=8, kv_heads=2,
                 intermediate=2816, vocab=4096, page_size=64, block=16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        dim = 128 if hidden // heads >= 128 else 64
        qkv = [heads * dim, kv_heads * dim, kv_heads * dim]

        def weight(*shape):
            return (torch.randn(*shape, device=device, generator=g) * shape[-1] ** -0.5).bfloat16()

        def norm():
            return dl.Norm((0.1 * torch.randn(hidden, device=device, generator=g)).bfloat16(), offset=1.0)

        def adapter(parts, cols):
            scale = torch.rand(adapters, device=device, generator=g)
            return dl.Adapters(weight(adapters, len(parts) * rank, cols), weight(adapters, sum(parts), rank),
                               scale=scale, parts=parts)

        self.rows, self.heads, self.kv_heads, self.dim, self.device = rows, heads, kv_heads, dim, device
        self.embed = weight(vocab, hidden) * hidden ** 0.5
        self.layers = [(norm(), weight(sum(qkv), hidden), adapter(qkv, hidden), weight(hidden, heads * dim),
                        adapter([hidden], heads * dim), norm(),
                        dl.interleave_gate_up(weight(intermediate, hidden), weight(intermediate, hidden)).contiguous(),
                        weight(hidden, intermediate)) for _ in range(layers)]
        self.last_norm, self.head = norm(), weight(vocab, hidden)
        self.caches = [dl.PagedKVCache.empty(pages, kv_heads, dim, page_size=page_size, block=block, device=device)
                       for _ in range(layers)]
        self.pool = dl.PagePool.empty(self.caches, rows, -(-max_len // page_size))
        angle = torch.outer(torch.arange(max_len, dtype=torch.float64),
                            1e6 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim))
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)
        shapes = [(m, n, k, dl.BF16) for m in (1, 16) for n, k in
                  ((sum(qkv), hidden), (hidden, heads * dim), (2 * intermediate, hidden), (hidden, intermediate),
                   (vocab, hidden))]
        self.workspace = dl.Workspace(max(
            dl.attention_workspace_bytes(rows, 16, heads, kv_heads, dim, max_q=16), dl.pages_workspace_bytes(self.pool),
            *(dl.adapters_workspace_bytes(16, a) for l in self.layers for a in (l[2], l[4])),
            *(dl.workspace_bytes(*s) for s in shapes)), device)

    def step(self, tokens, adapter, start, max_new):
        """Logits (fp32) of the new `tokens`, rows start[b] .. start[b + 1] of the pool's row b, which has room for
        them already; adapter[t] is token t's (all int32 tensors on the device)."""
        ws, pool = self.workspace, self.pool
        M, H, G, D = tokens.numel(), self.heads, self.kv_heads, self.dim
        norms = [l[0] for l in self.layers[1:]] + [self.last_norm]
        h = self.embed[tokens.long()]
        _, x = dl.block_norm(None, h, pre=self.layers[0][0])
        for (_, wqkv, aqkv, wo, ao, norm, wgu, wdown), cache, after in zip(self.layers, self.caches, norms):
            qkv = dl.linear_bf16(x, wqkv, workspace=ws)
            dl.linear_adapters(x, aqkv, adapter, qkv, out=qkv, workspace=ws)
            q, k, v = (t.view(M, -1, D) for t in qkv.split([H * D, G * D, G * D], dim=1))
            q = dl.kv_append(q, k, v, cache, pool.block_table, pool.seq_lens, start, max_q=max_new, cos=self.cos,
                             sin=self.sin)
            a = dl.attention_paged(q, cache, pool.block_table, pool.seq_lens, start, max_q=max_new, workspace=ws)
            a = a.view(M, H * D)
            o = dl.linear_bf16(a, wo, workspace=ws)
            dl.linear_adapters(a, ao, adapter, o, out=o, workspace=ws)
            h, x = dl.block_norm(o, h, pre=norm)
            y = dl.linear_bf16(dl.linear_swiglu(x, wgu, workspace=ws), wdown, workspace=ws)
            h, x = dl.block_norm(y, h, pre=after)
        logits = torch.empty(M, self.head.shape[0], device=self.device)
        dl.linear_bf16(x, self.head, out_f32=logits, workspace=ws)
        return logits

    def read(self, row, prompt, adapter):
        """A prompt (a list of ids) into the empty row `row`, 16 tokens at a time; its last token's logits."""
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=self.device)   # noqa: E731
        for i in range(0, len(prompt), 16):
            part = prompt[i:i + 16]
            done = dl.kv_reserve(self.pool, ints([row]), ints([len(part)]), workspace=self.workspace)
            if not int(done):
                raise RuntimeError("the pool has no room for the prompt")
            start = ints([0] * (row + 1) + [len(part)] * (self.rows - row))
            logits = self.step(ints(part), ints([adapter] * len(part)), start, len(part))
        return logits[-1]


def generate(model, prompts, adapters, n, *, branches=5, every=8, temperature=1.0, seed=0, graph=True):
    """The likeliest of `branches` continuations of n tokens for each prompt, and the mean log-probability of its
    tokens.  prompts: lists of ids; adapters: each one's adapter (-1: none)."""
    users, dev, pool, ws = len(prompts), model.device, model.pool, model.workspace
    R = users * branches
    if R != model.rows or R > 16:
        raise ValueError("users * branches must be the model's rows, at most 16, the linears' token limit")
    g = torch.Generator(device=dev).manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)   # noqa: E731
    heads = torch.arange(0, R, branches, dtype=torch.int32, device=dev)     # each user's first row
    rows = torch.arange(R, dtype=torch.int32, device=dev)
    logits = torch.stack([model.read(u * branches, p, a) for u, (p, a) in enumerate(zip(prompts, adapters))])
    logits = logits.repeat_interleave(branches, 0)
    served = [dl.kv_fork(pool, heads.repeat_interleave(branches), rows, workspace=ws)]
    own = ints(adapters).repeat_interleave(branches)
    ones, start, tokens = torch.ones_like(rows), ints(list(range(R + 1))), torch.zeros_like(rows)
    scores, texts = torch.zeros(R, device=dev), torch.zeros(R, 0, dtype=torch.int32, device=dev)
    replay, out = None, None

    def one():
        done = dl.kv_reserve(pool, rows, ones, workspace=ws)
        return done, model.step(tokens, own, start, 1)

    for i in range(n):
        logp = torch.log_softmax(logits / temperature, -1)
        picked = torch.multinomial(logp.exp(), 1, generator=g)
        scores += logp.gather(1, picked)[:, 0]
        texts = torch.cat([texts, picked.int()], 1)
        if i == n - 1:
            break
        if (i + 1) % every == 0:         # take all of a user's continuations up from the likeliest one
            best = heads + scores.view(users, branches).argmax(1).int()
            from_ = best.repeat_interleave(branches)
            dl.kv_free(pool, torch.where(rows == from_, -1, rows))      # (a row -1 is no row)
            done = dl.kv_fork(pool, from_, rows, workspace=ws)          # (a row is not forked to itself)
            served.append(done | (rows == from_).int())
            texts, scores = texts[from_.long()], scores[from_.long()]
        tokens.copy_(texts[:, -1])
        if graph and replay is None and i > 0:
            replay = torch.cuda.CUDAGraph()
            with torch.cuda.graph(replay):
                out = one()
        if replay is not None:
            replay.replay()
        else:
            out = one()
        done, logits = out[0].clone(), out[1]
        served.append(done)
    served[0] = served[0] | (rows == heads.repeat_interleave(branches)).int()
    if not bool(torch.stack(served).all()):
        raise RuntimeError("the pool ran out of pages")
    best = heads + scores.view(users, branches).argmax(1).int()
    return texts[best.long()].tolist(), (scores[best.long()] / n).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("users", 3), ("branches", 5), ("tokens", 48), ("every", 8), ("hidden", 1024), ("layers", 2),
                        ("heads", 8), ("kv-heads", 2), ("intermediate", 2816), ("vocab", 4096), ("rank", 16), ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--temperature", type=float, default=1.0)
    a = ap.parse_args()
    rows, length = a.users * a.branches, 40 + a.tokens
    model = Decoder(rows=rows, max_len=length, pages=rows * -(-length // 64), rank=a.rank, hidden=a.hidden,
                    layers=a.layers, heads=a.heads, kv_heads=a.kv_heads, intermediate=a.intermediate, vocab=a.vocab,
                    seed=a.seed)
    prompts = torch.randint(a.vocab, (a.users, 40), generator=torch.Generator().manual_seed(a.seed)).tolist()
    texts, scores = generate(model, prompts, [u % 5 - 1 for u in range(a.users)], a.tokens, branches=a.branches,
                             every=a.every, temperature=a.temperature, seed=a.seed)
    for t, s in zip(texts, scores):
        print(f"{s:.3f}", t)
    live = int(dl.kv_compact(model.pool))
    print(f"{live} of {model.pool.num_pages} pages in use")


if __name__ == "__main__":
    main()
