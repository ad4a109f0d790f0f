"""Measured cases of what a decode step of many requests does around its linear layers.

  norm      the end of one block and the start of the next: the block's output is normalised
            (or not), gated and scaled, added to the residual stream, and the stream's norm is
            the next linear's input (block_norm);
  adapters  low-rank adapters beside a shared projection, another one for each token
            (linear_adapters);
  beam      one step of sampling several continuations: the rows that lost give their cache
            pages back, the winners are forked into them, and the new rows get room for their next
            tokens (kv_free, kv_fork, kv_reserve);
  compact   the pages that are in use move to the front of the pool (kv_compact).

``run`` computes an operator in its plain form with elementary torch operations in 32 bits, or,
where ``own`` is true, by the framework's calls.  ``exact`` gives norms and adapters in 64 bits; the
cache's operators move codes and whole numbers.
"""
from __future__ import annotations

import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64

# The largest of each kind, which bound what is drawn.
_NORM_MOST = 16384 * 8192               # elements of the stream
_ADAPTER_MOST = 4096 * 10240            # outputs
_POOL_MOST = 2048 * 8 * 8 * 64 * 128    # key codes of all layers


def _norm(name, rows, dim, post="none", pre="rms", gate="none", act=False, y="bf16", h="bf16", bias=False,
          offset=0.0, scale=1.0):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "post": post, "pre": pre, "gate": gate,
            "act": act, "y": y, "h": h, "bias": bias, "offset": offset, "scale": scale}


def _adapters(name, tokens, K, N, rank, num, parts="one", base="bf16", mixed=True, f32=False, ragged=False):
    return {"name": name, "op": "adapters", "tokens": tokens, "K": K, "N": N, "rank": rank, "num": num,
            "parts": parts, "base": base, "mixed": mixed, "f32": f32, "ragged": ragged}


def _beam(name, users, width, length, layers, spare, kv_heads=8, dim=128, page=64, block=16, add=1):
    return {"name": name, "op": "beam", "users": users, "width": width, "length": length, "layers": layers,
            "spare": spare, "kv_heads": kv_heads, "dim": dim, "page": page, "block": block, "add": add}


def _compact(name, pages, rows, layers, used, kv_heads=8, dim=128, page=64, block=16):
    return {"name": name, "op": "compact", "pages": pages, "rows": rows, "layers": layers, "used": used,
            "kv_heads": kv_heads, "dim": dim, "page": page, "block": block}


def listed():
    return [
        # one token between two linears of the 8192-wide decoder, the stream in fp32: a latency
        _norm("norm_one_token", 1, 8192, h="fp32"),
        # the 16 tokens of the widest decode step, norms before and after the block, weights stored
        # as differences from 1, a gate and a residual scale
        _norm("norm_sandwich_16", 16, 8192, post="rms", gate="channel", offset=1.0, scale=0.25),
        # an odd width, centred norms with biases, the block's output in fp32, a gate for each element
        _norm("norm_odd_gated", 999, 1537, post="layer", pre="layer", gate="full", act=True, y="fp32", bias=True),
        # prompts: the largest
        _norm("norm_prompts", 16384, 8192),
        # one request's token through the fused 8192 -> 10240 projection of queries, keys and values
        _adapters("adapters_one_token", 1, 8192, 10240, 16, 32, parts="qkv"),
        # a full decode step of 16 requests through the 29568 -> 8192 projection, fp32 results
        _adapters("adapters_step_16", 16, 29568, 8192, 32, 64, base="fp32", f32=True),
        # a large batch of requests in any order, ranks of many sizes, some without an adapter
        _adapters("adapters_batch_256", 256, 8192, 8192, 16, 64, ragged=True),
        # prompts of four requests, one after the other: the largest
        _adapters("adapters_prompts", 4096, 8192, 10240, 64, 8, parts="qkv", mixed=False),
        # one user, four continuations, all 80 layers
        _beam("beam_one_user", 1, 4, 1000, 80, 8),
        # a batch of users with five continuations each, one stage's 8 layers
        _beam("beam_batch", 32, 5, 3001, 8, 100),
        # a pool that has emptied out, all 80 layers
        _compact("compact_small", 80, 6, 80, 0.3),
        # a large pool half in use: the largest
        _compact("compact_large", 2048, 64, 8, 0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "adapters", "adapters", "adapters", "beam", "compact"])
    if op == "norm":
        dim = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            dim = -(-dim // 64) * 64
        rows = min(_log(rng, 1, 16384), _NORM_MOST // dim)
        post = rng.choice(["none", "none", "rms", "layer"])
        return {"op": op, "rows": rows, "dim": dim, "post": post, "pre": rng.choice(["rms", "rms", "layer"]),
                "gate": rng.choice(["none", "channel", "row", "full"]), "act": rng.random() < 0.5,
                "y": rng.choice(["bf16", "fp32"]), "h": rng.choice(["bf16", "fp32"]),
                "bias": rng.random() < 0.5, "offset": rng.choice([0.0, 1.0]), "scale": rng.choice([1.0, 0.5])}
    if op == "adapters":
        K, rank, num = 8 * _log(rng, 32, 3696), rng.choice([8, 16, 24, 32, 64, 128]), _log(rng, 1, 64)
        tokens, parts = _log(rng, 1, 4096), rng.choice(["one", "one", "qkv", "two"])
        N = _log(rng, 200, 29568)
        if parts != "one":
            N = 96 * max(2, N // 96)
        while tokens > 1 and (tokens * N > _ADAPTER_MOST or tokens * (K + N) * rank > 4096 * 18432 * 64):
            tokens = (tokens + 1) // 2
        return {"op": op, "tokens": tokens, "K": K, "N": N, "rank": rank, "num": num, "parts": parts,
                "base": rng.choice(["bf16", "fp32", "none"]), "mixed": rng.random() < 0.6,
                "f32": rng.random() < 0.25, "ragged": rng.random() < 0.4}
    case = {"op": op, "kv_heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]),
            "page": rng.choice([16, 32, 64, 128]), "layers": _log(rng, 1, 80)}
    case["block"] = rng.choice([4, 16, case["page"]])
    size = case["layers"] * case["kv_heads"] * case["dim"] * case["page"]      # codes of a page
    most = max(24, min(4096, _POOL_MOST // size))
    if op == "compact":
        return {**case, "pages": _log(rng, 16, most), "rows": _log(rng, 2, 64), "used": rng.uniform(0.1, 0.95)}
    width, users, length = rng.randint(2, 8), _log(rng, 1, 32), _log(rng, 1, 4096)
    add = rng.choice([1, 1, 4, 40])

    def pages():
        return users * (-(-length // case["page"]) + width * (3 + add // case["page"]))

    while pages() > most and length > 1:
        length //= 2
    while pages() > most and users > 1:
        users //= 2
    return {**case, "users": users, "width": width, "length": length, "add": add, "spare": rng.randint(0, 20)}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "adapters": _prepare_adapters, "beam": _prepare_beam,
            "compact": _prepare_compact}[case["op"]](case, gen, seed)


def _kind(name):
    return {"bf16": BF16, "fp32": F32}[name]


def _prepare_norm(case, gen, seed):
    T, D = case["rows"], case["dim"]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    channels = torch.exp(0.5 * randn(D))              # channels of unequal size
    s = {"op": "norm", "post": case["post"], "pre": case["pre"], "offset": case["offset"], "scale": case["scale"],
         "act": case["act"], "eps": 1e-6,
         "y": (0.7 * randn(T, D) * channels + 0.1).to(_kind(case["y"])),
         "h": (3.0 * randn(T, D) * channels - 0.2).to(_kind(case["h"]))}
    for n in ("post", "pre"):
        w, b = (1.0 + 0.1 * randn(D)) - case["offset"], 0.1 * randn(D)
        s[n + "_w"] = w.to(BF16)
        s[n + "_b"] = b.to(BF16) if case["bias"] else None
    shape = {"none": None, "channel": (D,), "row": (T, 1), "full": (T, D)}[case["gate"]]
    s["gate"] = None if shape is None else (0.5 + randn(*shape)).to(BF16)
    if own:
        import weight_streaming_skinny_gb300 as dl
        for n in ("post", "pre"):
            s[n + "_norm"] = None if case[n] == "none" else dl.Norm(
                s[n + "_w"], s[n + "_b"], kind=case[n], eps=s["eps"], offset=case["offset"])
    return s


def _columns(case):
    """Columns of the projections that lie side by side in N."""
    N = case["N"]
    if case["parts"] == "qkv":
        side = max(16, N // 10 // 16 * 16)
        return [N - 2 * side, side, side]
    return [N // 2, N - N // 2] if case["parts"] == "two" else [N]


def _prepare_adapters(case, gen, seed):
    T, K, N, R, num = (case[n] for n in ("tokens", "K", "N", "rank", "num"))
    cpu = torch.Generator().manual_seed(seed)
    cols = _columns(case)
    x = torch.randn(T, K, device="cuda", generator=gen)
    x *= torch.exp(0.3 * torch.randn(T, 1, device="cuda", generator=gen))
    a = torch.randn(num, len(cols) * R, K, device="cuda", generator=gen) * K ** -0.5
    b = torch.randn(num, N, R, device="cuda", generator=gen) * (0.5 * R ** -0.5)
    base = torch.randn(T, N, device="cuda", generator=gen)
    if case["mixed"]:       # any order; one token in ten without an adapter
        index = torch.randint(num, (T,), generator=cpu)
        index[torch.rand(T, generator=cpu) < 0.1] = -1
        if T == 1:
            index[0] = int(torch.randint(num, (1,), generator=cpu))
    else:                   # four requests, one after the other
        which = torch.randint(num, (4,), generator=cpu)
        index = which[(torch.arange(T) * 4) // max(T, 1)]
    # what lies past an adapter's rank is what was there before
    ranks = torch.randint(1, R + 1, (num,), generator=cpu) if case["ragged"] else torch.full((num,), R)
    s = {"op": "adapters", "x": x.to(BF16), "a": a.to(BF16), "b": b.to(BF16), "cols": cols, "f32": case["f32"],
         "scale": (0.5 + 1.5 * torch.rand(num, generator=cpu)).cuda(), "index": index.int().cuda(),
         "ranks": ranks.int().cuda(), "base": None if case["base"] == "none" else base.to(_kind(case["base"]))}
    if own:
        import weight_streaming_skinny_gb300 as dl
        s["adapters"] = dl.Adapters(s["a"], s["b"], scale=s["scale"], ranks=s["ranks"], parts=cols)
        s["workspace"] = dl.Workspace(dl.adapters_workspace_bytes(T, s["adapters"]))
        if case["f32"]:
            s["out_f32"] = torch.empty(T, N, device="cuda")
    return s


def _pool(case, pages, gen, s):
    """Caches of all layers with random codes (no NaN), each layer a view of one buffer."""
    L, H, D, P, blk = (case[n] for n in ("layers", "kv_heads", "dim", "page", "block"))
    for n in ("k", "v"):
        c = torch.randint(0, 256, (L, pages, H, P, D), dtype=torch.uint8, device="cuda", generator=gen)
        s[n] = c.masked_fill_((c & 127) == 127, 3)
        s[n + "_scale"] = torch.exp2(torch.randint(-12, -2, (L, pages, H, P // blk), device="cuda",
                                                   generator=gen).float())
    s["page"], s["block"] = P, blk
    if own:
        import weight_streaming_skinny_gb300 as dl
        caches = [dl.PagedKVCache(s["k"][i], s["v"][i], s["k_scale"][i], s["v_scale"][i]) for i in range(L)]
        s["pool"] = dl.PagePool(caches, s["table"], s["lens"], s["refs"])
        s["workspace"] = dl.Workspace(dl.pages_workspace_bytes(s["pool"]))
    return s


def _prepare_beam(case, gen, seed):
    """Users of `width` rows each: a user's rows share the full pages of their common start and have
    their own pages from there on.  Half of each user's rows (rounded up, but one) lose."""
    U, W, P, add = case["users"], case["width"], case["page"], case["add"]
    cpu = torch.Generator().manual_seed(17)
    shape = torch.randint(max(1, case["length"] // 2), case["length"] + 1, (U,), generator=cpu).tolist()
    shape[-1] = case["length"]
    shape = [shape[i] for i in torch.randperm(U, generator=torch.Generator().manual_seed(seed)).tolist()]
    cols = max(shape) // P + 4 + (add + P) // P
    pages = sum(n // P + W * (3 + add // P) for n in shape) + case["spare"]
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 1)).tolist()
    table = torch.full((U * W, cols), -1, dtype=torch.int32)
    refs, lens = torch.zeros(pages, dtype=torch.int32), torch.zeros(U * W, dtype=torch.int32)
    parents, children = [], []
    lose = max(1, min(W - 1, (W + 1) // 2))
    extra = torch.randint(0, P, (U, W), generator=torch.Generator().manual_seed(seed + 2))
    for u, n in enumerate(shape):
        shared = [order.pop() for _ in range(n // P)]
        for w in range(W):
            row, length = u * W + w, n + int(extra[u, w])
            mine = shared + [order.pop() for _ in range(-(-length // P) - len(shared))]
            table[row, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            refs[torch.tensor(mine)] += 1
            lens[row] = length
        for i in range(lose):           # the first rows of a user win in turn
            parents.append(u * W + i % (W - lose))
            children.append(u * W + W - 1 - i)
    s = {"op": "beam", "table": table.cuda(), "lens": lens.cuda(), "refs": refs.cuda()}
    for n, v in (("parents", parents), ("children", children), ("add", [add] * len(children))):
        s[n] = torch.tensor(v, dtype=torch.int32, device="cuda")
    return _pool(case, pages, gen, s)


def _prepare_compact(case, gen, seed):
    """`rows` sequences over the used pages in any order; one in eight starts as another one does."""
    pages, rows, P = case["pages"], case["rows"], case["page"]
    used = max(1, min(pages - 1, int(pages * case["used"])))
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:used].tolist()
    each = max(1, used // rows)
    cols = each + used % rows + 2 + each
    table = torch.full((rows, cols), -1, dtype=torch.int32)
    refs, lens = torch.zeros(pages, dtype=torch.int32), torch.zeros(rows, dtype=torch.int32)
    first = []
    for r in range(rows):
        n = min(len(order), each + (used % rows if r == rows - 1 else 0))
        mine = (first if r % 8 == 7 else []) + [order.pop() for _ in range(n)]
        if r == 0:
            first = mine
        if not mine:
            continue
        table[r, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
        refs[torch.tensor(mine)] += 1
        lens[r] = len(mine) * P - r % P
    s = {"op": "compact", "table": table.cuda(), "lens": lens.cuda(), "refs": refs.cuda()}
    # the pool as it is found: a pass starts from it again
    s["table_found"], s["refs_found"] = s["table"].clone(), s["refs"].clone()
    return _pool(case, pages, gen, s)


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return {"norm": _own_norm, "adapters": _own_adapters, "beam": _own_beam, "compact": _own_compact}[s["op"]](s)
    return {"norm": _plain_norm, "adapters": _plain_adapters, "beam": _plain_beam,
            "compact": _plain_compact}[s["op"]](s)


def _own_norm(s):
    import weight_streaming_skinny_gb300 as dl
    h, x = dl.block_norm(s["y"], s["h"], post=s["post_norm"], pre=s["pre_norm"], gate=s["gate"],
                         gate_act="sigmoid" if s["act"] else None, scale=s["scale"])
    return {"h": h, "x": x}


def _own_adapters(s):
    import weight_streaming_skinny_gb300 as dl
    out32 = s.get("out_f32")
    out = dl.linear_adapters(s["x"], s["adapters"], s["index"], s["base"], out_f32=out32, workspace=s["workspace"])
    return {"out": out} if out32 is None else {"out": out, "out_f32": out32}


def _own_beam(s):
    import weight_streaming_skinny_gb300 as dl
    dl.kv_free(s["pool"], s["children"])
    forked = dl.kv_fork(s["pool"], s["parents"], s["children"], workspace=s["workspace"])
    grown = dl.kv_reserve(s["pool"], s["children"], s["add"], workspace=s["workspace"])
    return _pool_out(s, forked=forked, grown=grown)


def _own_compact(s):
    import weight_streaming_skinny_gb300 as dl
    s["table"].copy_(s["table_found"])
    s["refs"].copy_(s["refs_found"])
    return _pool_out(s, live=dl.kv_compact(s["pool"], workspace=s["workspace"]))


def _pool_out(s, **more):
    f8 = torch.float8_e4m3fn
    return {"k": s["k"].view(f8), "v": s["v"].view(f8), "k_scale": s["k_scale"], "v_scale": s["v_scale"],
            "table": s["table"], "lens": s["lens"], "refs": s["refs"], **more}


def _normed(x, kind, w, b, offset, eps):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * (w.to(x.dtype) + offset)
    return x if b is None else x + b.to(x.dtype)


def _plain_norm(s):
    u = _normed(s["y"].float(), s["post"], s["post_w"], s["post_b"], s["offset"], s["eps"])
    if s["gate"] is not None:
        g = s["gate"].float()
        u = u * (1 / (1 + torch.exp(-g)) if s["act"] else g)
    r = s["h"].float() + s["scale"] * u
    x = _normed(r, s["pre"], s["pre_w"], s["pre_b"], s["offset"], s["eps"])
    return {"h": r.to(s["h"].dtype), "x": x.to(BF16)}


def _plain_adapters(s):
    """Every adapter's first product for every token, the others' then left out."""
    x, a, b, cols = s["x"].float(), s["a"], s["b"], s["cols"]
    num, N, R = b.shape
    T, S = x.shape[0], len(cols)
    each = torch.arange(num, device=x.device)
    mine = (s["index"][:, None] == each)[:, :, None, None]                              # [T, num, 1, 1]
    within = (torch.arange(R, device=x.device) < s["ranks"][:, None])                   # [num, R]
    low = torch.matmul(x, a.float().view(num * S * R, -1).t()).view(T, num, S, R) * s["scale"][:, None, None]
    low = torch.where(mine & within[:, None], low, 0.0)
    up = torch.where(within[:, None], b.float(), 0.0).transpose(1, 2).reshape(num * R, N)
    first = [sum(cols[:i]) for i in range(S)]
    out = torch.cat([torch.matmul(low[:, :, i].reshape(T, num * R), up[:, f:f + c])
                     for i, (f, c) in enumerate(zip(first, cols))], 1)
    if s["base"] is not None:
        out = s["base"].float() + out
    return {"out": out.to(BF16), "out_f32": out} if s["f32"] else {"out": out.to(BF16)}


def _pages_of(s, rows):
    """(page of each column, whether it is used) of `rows`."""
    at = torch.arange(s["table"].shape[1], device="cuda")
    used = at < ((s["lens"][rows] + s["page"] - 1) // s["page"])[:, None]
    return s["table"][rows].long(), used


def _take(refs, need):
    """The lowest free pages for each of `need`, in order: (sorted page numbers, first, granted)."""
    free = torch.argsort((refs > 0).int(), stable=True)
    last = torch.cumsum(need, 0)
    return free, last - need, (need == 0) | (last <= (refs == 0).sum())


def _plain_beam(s):
    refs, table, lens, P, blk = s["refs"], s["table"], s["lens"], s["page"], s["block"]
    kids, par, cols = s["children"].long(), s["parents"].long(), s["table"].shape[1]
    at = torch.arange(cols, device="cuda")
    # give back
    page, used = _pages_of(s, kids)
    refs.index_add_(0, page.clamp(min=0).view(-1), -used.int().view(-1))
    lens[kids] = 0
    # fork: full pages are shared, a page that is begun is copied as far as it is filled
    n, (page, used) = lens[par], _pages_of(s, par)
    tail = n % P
    need = (tail > 0).int()
    free, first, ok = _take(refs, need)
    fresh = free[first.clamp(max=refs.numel() - 1)]
    full = used & (at < (n // P)[:, None]) & ok[:, None]
    refs.index_add_(0, page.clamp(min=0).view(-1), full.int().view(-1))
    copies = ok & (need > 0)
    last = page.gather(1, (n // P).clamp(max=cols - 1)[:, None].long())[:, 0]
    held = torch.arange(P, device="cuda") < tail[:, None]
    src, dst = last[copies], fresh[copies]
    keep = held[copies][:, None, :, None]
    blocks = torch.arange(P // blk, device="cuda") * blk < tail[copies][:, None]
    for name in ("k", "v"):
        s[name][:, dst] = torch.where(keep, s[name][:, src], s[name][:, dst])
        c = s[name + "_scale"]
        c[:, dst] = torch.where(blocks[:, None], c[:, src], c[:, dst])
    refs.index_add_(0, fresh, copies.int())
    new = torch.where(at == (n // P)[:, None], fresh[:, None], page).int()
    table[kids] = torch.where(used & ok[:, None], new, table[kids])
    lens[kids] = torch.where(ok, n, 0)
    # room for the next tokens
    n, add = lens[kids], s["add"]
    need = (n + add + P - 1) // P - (n + P - 1) // P
    free, first, grown = _take(refs, need)
    begin = (n + P - 1) // P
    mine = (at >= begin[:, None]) & (at < (begin + need)[:, None]) & grown[:, None]
    fresh = free[(first[:, None] + at - begin[:, None]).clamp(0, refs.numel() - 1).long()]
    refs.index_add_(0, fresh.view(-1), mine.int().view(-1))
    table[kids] = torch.where(mine, fresh.int(), table[kids])
    lens[kids] = torch.where(grown, n + add, n)
    return _pool_out(s, forked=ok.int(), grown=grown.int())


def _plain_compact(s):
    s["table"].copy_(s["table_found"])
    s["refs"].copy_(s["refs_found"])
    refs, table = s["refs"], s["table"]
    N = refs.numel()
    at, live = torch.arange(N, device="cuda"), (refs > 0).sum()
    src = at[(refs > 0) & (at >= live)]
    dst = at[(refs == 0) & (at < live)]
    for name in ("k", "v", "k_scale", "v_scale"):
        s[name][:, dst] = s[name][:, src]
    to = at.clone()
    to[src] = dst
    page, used = _pages_of(s, slice(None))
    table.copy_(torch.where(used, to[page.clamp(min=0)], page).int())
    refs[dst] = refs[src]
    refs[src] = 0
    return _pool_out(s, live=live.int().view(1))


# ------------------------------------------------------------------ cost and 64-bit values

def work(case):
    if case["op"] == "norm":
        n, D = case["rows"] * case["dim"], case["dim"]
        size = {"bf16": 2, "fp32": 4}
        gate = {"none": 0, "channel": 2 * D, "row": 2 * case["rows"], "full": 2 * n}[case["gate"]]
        weights = 2 * D * (1 + case["bias"]) * (1 + (case["post"] != "none"))
        return {"bytes": n * (size[case["y"]] + 2 * size[case["h"]] + 2) + gate + weights, "flops": 12 * n}
    if case["op"] == "adapters":
        T, K, N, R, num = (case[n] for n in ("tokens", "K", "N", "rank", "num"))
        S = len(_columns(case))
        users = 0.9 * T if case["mixed"] and T > 1 else T
        seen = num * (1 - (1 - 1 / num) ** (users if case["mixed"] else 4)) if num > 1 else 1
        seen = min(seen, T)
        r = (R + 1) / 2 if case["ragged"] else R
        size = {"bf16": 2, "fp32": 4, "none": 0}[case["base"]] + 2 + (4 if case["f32"] else 0)
        return {"bytes": 2 * T * K + 2 * seen * r * (S * K + N) + T * N * size,
                "flops": 2 * users * r * (S * K + N)}
    code = case["kv_heads"] * case["dim"] * case["page"] + 4 * case["kv_heads"] * case["page"] // case["block"]
    page = 2 * code * case["layers"]
    if case["op"] == "compact":
        used, n = max(1, min(case["pages"] - 1, int(case["pages"] * case["used"]))), case["pages"]
        moved = used * (n - used) / n
        return {"bytes": 2 * moved * page + 8 * n + 8 * used, "flops": n}
    U, W = case["users"], case["width"]
    n = U * max(1, min(W - 1, (W + 1) // 2))
    held = n * (0.75 * case["length"] / case["page"] + 1)
    # a page that is begun is half full on the average
    return {"bytes": n * page + 8 * held + 4 * n * 5, "flops": held}


def _normed64(x, kind, w, b, offset, eps):
    if kind == "none":
        return x
    D = x.shape[-1]
    if kind == "layer":
        x = x - (x.sum(-1) / D)[:, None]
    x = x / torch.sqrt((x.square().sum(-1) / D + eps))[:, None]
    x = x * (offset + w.double())
    return x + b.double() if b is not None else x


def exact(case, seed):
    if case["op"] in ("beam", "compact"):
        return None                     # codes and whole numbers only
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = torch.empty(s["h"].shape, dtype=F64, device="cuda")
        x = torch.empty_like(h)
        for i in range(0, case["rows"], 2048):
            at = slice(i, i + 2048)
            u = _normed64(s["y"][at].double(), case["post"], s["post_w"], s["post_b"], case["offset"], s["eps"])
            if s["gate"] is not None:
                g = (s["gate"] if case["gate"] == "channel" else s["gate"][at]).double()
                u = u * (torch.sigmoid(g) if case["act"] else g)
            h[at] = s["h"][at].double() + case["scale"] * u
            x[at] = _normed64(h[at], case["pre"], s["pre_w"], s["pre_b"], case["offset"], s["eps"])
        return {"h": h, "x": x}
    T, N, R = case["tokens"], case["N"], case["rank"]
    out = torch.zeros(T, N, dtype=F64, device="cuda") if s["base"] is None else s["base"].double()
    for i in sorted(set(s["index"].tolist()) - {-1}):
        rows = (s["index"] == i).nonzero()[:, 0]
        r, c0 = int(s["ranks"][i]), 0
        for part, c in enumerate(s["cols"]):
            low = s["x"][rows].double() @ s["a"][i, part * R:part * R + r].double().t()
            out[rows, c0:c0 + c] += s["scale"][i].double() * (low @ s["b"][i, c0:c0 + c, :r].double().t())
            c0 += c
    return {"out": out, "out_f32": out.clone()} if case["f32"] else {"out": out}
