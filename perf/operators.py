"""Measured cases of the cached-attention operators: kv_append, attention_paged, verify_draft.

One step of speculative decoding runs, next to the linear layers, three
operators on state that the linears do not touch:

  append  rotates the new tokens' queries and keys by their positions and
          writes keys and values into a paged cache of e4m3 codes with one fp32
          scale for each block of tokens and head;
  attn    attends from the new tokens (one for plain decoding, several to
          verify a draft) to that cache;
  verify  accepts a prefix of the drafted tokens and draws the next token from
          given random numbers.

``run`` computes an operator in its plain form with elementary torch
operations in 32 bits, or, where ``own`` is true, by the framework's calls.
``exact`` gives the attention output and the rotated queries in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE_EXP = -40        # the smallest scale an append writes is 2^-40
WEIGHT_BITS = 44           # verify: probabilities as whole multiples of 2^-44

# The largest listed attention case: 64 sequences of up to 16384 tokens, 8 key/value heads of 128.
_CAP_BYTES = 64 * 16384 * 8 * 128 * 2
_CAP_FLOPS = 4 * 64 * 16384 * 64 * 128


def _attn(name, batch, q, length, heads=64, kv_heads=8, dim=128, page=64, block=16, ragged=True):
    return {"name": name, "op": "attn", "batch": batch, "q": q, "length": length, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "block": block, "ragged": ragged}


def _append(name, batch, q, past, heads=64, kv_heads=8, dim=128, page=64, block=16, ragged=True):
    return {"name": name, "op": "append", "batch": batch, "q": q, "past": past, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "block": block, "ragged": ragged}


def _verify(name, batch, drafts, vocab, kind="fp32", draft_probs=True):
    return {"name": name, "op": "verify", "batch": batch, "drafts": drafts, "vocab": vocab,
            "kind": kind, "draft_probs": draft_probs}


def listed():
    return [
        # one user, one token, a short chat: nothing but latency (64 query heads on 8 key/value
        # heads of 128, as behind the 8192 -> 10240 QKV projection)
        _attn("attn_one_user_short", 1, 1, 500, ragged=False),
        # one user with a long document: the work has to be split along the cache
        _attn("attn_one_user_long", 1, 1, 30011, ragged=False),
        # ordinary batched decoding, ragged lengths
        _attn("attn_batch_decode", 32, 1, 4096),
        # a verify step of 6 tokens over a batch, ragged lengths and drafts
        _attn("attn_batch_verify", 16, 6, 8192),
        # 16 tokens a sequence, the most one decode step of the framework takes
        _attn("attn_verify_16", 4, 16, 32768, ragged=False),
        # a small model's heads: 3 query heads on each of 8 key/value heads of 64, small pages
        _attn("attn_dim64_odd", 24, 3, 2049, heads=24, kv_heads=8, dim=64, page=16, block=16),
        # the largest: a full server at long contexts
        _attn("attn_largest", 64, 1, 16384, page=128, block=32),
        # one token of one user appended inside a block that is already begun
        _append("append_one_token", 1, 1, 777, ragged=False),
        # a batch of verify steps appended
        _append("append_batch_verify", 48, 6, 1000),
        # prompts written to the cache
        _append("append_prompts", 4, 4096, 300),
        # one user's draft of 5 tokens against the 152064-token vocabulary
        _verify("verify_one_user", 1, 5, 152064),
        # a batch of drafts
        _verify("verify_batch", 48, 5, 152064),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "verify"])
    if op == "verify":
        drafts = rng.randint(1, 15)
        vocab = _log(rng, 1000, 152064)
        batch = _log(rng, 1, 64)
        while batch > 1 and batch * (drafts + 1) * vocab > 48 * 6 * 152064:
            batch //= 2
        return {"op": op, "batch": batch, "drafts": drafts, "vocab": vocab,
                "kind": rng.choice(["fp32", "fp32", "bf16"]), "draft_probs": rng.random() < 0.75}
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([4, 16, page])
    case = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page,
            "block": block, "ragged": rng.random() < 0.7}
    if op == "append":
        q = _log(rng, 1, 4096)
        batch = _log(rng, 1, 64)
        while batch > 1 and batch * q > 16384:
            batch //= 2
        return {**case, "batch": batch, "q": q, "past": _log(rng, 1, 2000)}
    q = rng.choice([1, 1, rng.randint(2, 16)])
    length = max(q, _log(rng, 1, 32768))
    batch = _log(rng, 1, 64)
    while batch > 1 and (batch * length * kv_heads * dim * 2 > _CAP_BYTES
                         or 4 * batch * length * kv_heads * group * q * dim > _CAP_FLOPS):
        batch //= 2
    return {**case, "batch": batch, "q": q, "length": length}


# ------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """Tokens in the cache after the step and new tokens, of each sequence (host lists). Ragged
    sizes are the case's own, so that outputs of every seed have the same shapes; the seed says
    which sequence has which."""
    g = torch.Generator().manual_seed(17)
    B, q = case["batch"], case["q"]
    whole = case["past"] if case["op"] == "append" else case["length"]
    news, held = [q] * B, [whole] * B
    if case["ragged"]:
        news = torch.randint(max(1, q // 2), q + 1, (B,), generator=g).tolist()
        held = torch.randint(max(1, whole // 2), whole + 1, (B,), generator=g).tolist()
        news[0], held[-1] = q, whole
    lens = [h + n if case["op"] == "append" else max(h, n) for h, n in zip(held, news)]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
    return [lens[i] for i in order], [news[i] for i in order]


def _cache(case, pages, gen, dev):
    """Random keys or values as an append stores them: e4m3 codes [pages, kv_heads, page, dim]
    with the smallest power-of-two scale that holds each block."""
    H, D, P, blk = case["kv_heads"], case["dim"], case["page"], case["block"]
    x = torch.randn(pages, H, P // blk, blk, D, device=dev, generator=gen)
    x *= torch.exp(0.5 * torch.randn(1, H, 1, 1, D, device=dev, generator=gen))   # channels of unequal size
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(3, 4)) / E4M3_MAX)))
    x /= scale[..., None, None]
    codes = x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(pages, H, P, D).view(torch.uint8), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "verify":
        return _prepare_verify(case, gen, dev)
    lens, news = _lengths(case, seed)
    B, Hq, Hkv, D, P = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    cols = max(-(-n // P) for n in lens) + 1
    pages = sum(-(-n // P) for n in lens) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 1)).tolist()
    table = torch.zeros(B, cols, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // P)
        table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    k, ks = _cache(case, pages, gen, dev)
    v, vs = _cache(case, pages, gen, dev)
    T = sum(news)
    start = torch.zeros(B + 1, dtype=torch.int32)
    start[1:] = torch.cumsum(torch.tensor(news), 0)
    # the QKV projection's output: queries, keys and values of a token side by side
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, device=dev, generator=gen)
    qkv *= torch.exp(0.3 * torch.randn(T, 1, device=dev, generator=gen))
    qkv = qkv.to(torch.bfloat16)
    s = {"op": case["op"], "k": k, "v": v, "k_scale": ks, "v_scale": vs, "block": case["block"],
         "table": table.to(dev), "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "start": start.to(dev), "max_q": max(news), "max_len": max(lens),
         "q": qkv[:, :Hq * D].view(T, Hq, D),
         "new_k": qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
         "new_v": qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)}
    if case["op"] == "append":
        angle = torch.outer(torch.arange(max(lens), dtype=torch.float64),
                            1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D))
        s["cos"] = torch.cos(angle).float().to(dev)
        s["sin"] = torch.sin(angle).float().to(dev)
    else:
        s["q"] = s["q"].contiguous()
    if own:
        import weight_streaming_skinny_gb300 as dl
        s["cache"] = dl.PagedKVCache(k, v, ks, vs)
        if case["op"] == "attn":
            s["workspace"] = dl.Workspace(dl.attention_workspace_bytes(
                B, T, Hq, Hkv, D, max_q=s["max_q"]))
    return s


def _prepare_verify(case, gen, dev):
    B, S, V = case["batch"], case["drafts"], case["vocab"]
    kind = torch.float32 if case["kind"] == "fp32" else torch.bfloat16
    logits = 2.5 * torch.randn(B, S + 1, V, device=dev, generator=gen)
    logits += 6.0 * (torch.rand(B, S + 1, V, device=dev, generator=gen) < 8.0 / V)   # a few likely tokens
    target = torch.softmax(logits, -1)
    guess = torch.softmax(logits[:, :S] + 0.3 * torch.randn(B, S, V, device=dev, generator=gen), -1)
    pick = torch.rand(B, S, 1, device=dev, generator=gen, dtype=torch.float64)
    drafts = torch.searchsorted(torch.cumsum(guess.double(), -1), pick).clamp_(max=V - 1)[..., 0].int()
    return {"op": "verify", "drafts": drafts, "target": target.to(kind),
            "guess": guess.to(kind) if case["draft_probs"] else None,
            "u": torch.rand(B, S, device=dev, generator=gen),
            "u_next": torch.rand(B, device=dev, generator=gen)}


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"append": _plain_append, "attn": _plain_attn, "verify": _plain_verify}[s["op"]](s)


def _run_own(s):
    import weight_streaming_skinny_gb300 as dl
    if s["op"] == "attn":
        return dl.attention_paged(s["q"], s["cache"], s["table"], s["lens"], s["start"],
                                  max_q=s["max_q"], workspace=s["workspace"])
    if s["op"] == "append":
        q = dl.kv_append(s["q"], s["new_k"], s["new_v"], s["cache"], s["table"], s["lens"],
                         s["start"], max_q=s["max_q"], cos=s["cos"], sin=s["sin"])
        return _appended(s, q)
    tokens, count = dl.verify_draft(s["drafts"], s["target"], s["u"], s["u_next"],
                                    draft_probs=s["guess"])
    return {"tokens": tokens, "count": count}


def _appended(s, q):
    f8 = torch.float8_e4m3fn
    return {"q": q, "k": s["k"].view(f8), "v": s["v"].view(f8), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _plain_attn(s):
    q, start, lens, L, Q = s["q"], s["start"].long(), s["lens"].long(), s["max_len"], s["max_q"]
    T, Hq, D = q.shape
    pages, Hkv, P, _ = s["k"].shape
    B, blk, dev = lens.numel(), s["block"], q.device
    cols = -(-L // P)
    table = s["table"][:, :cols].long()

    def gathered(codes, scale):           # [B, Hkv, cols * P, D] in fp32
        x = codes.view(torch.float8_e4m3fn)[table].float().view(B, cols, Hkv, P // blk, blk, D)
        x = x * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4, 5).reshape(B, Hkv, cols * P, D)

    i = torch.arange(Q, device=dev)
    news = start[1:] - start[:-1]
    token = (start[:-1, None] + i).clamp(max=T - 1)                       # [B, Q]
    qp = q[token].float().view(B, Q, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = torch.matmul(qp, gathered(s["k"], s["k_scale"]).transpose(-1, -2)) * (D ** -0.5)
    score = score.view(B, Hkv, Hq // Hkv, Q, cols * P)
    seen = torch.arange(cols * P, device=dev) <= (lens - news)[:, None, None] + i[:, None]
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p.view(B, Hkv, -1, cols * P), gathered(s["v"], s["v_scale"]))
    o = o.view(B, Hkv, Hq // Hkv, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)
    b = torch.searchsorted(start, torch.arange(T, device=dev), right=True) - 1
    return o[b, torch.arange(T, device=dev) - start[b]].to(torch.bfloat16)


def _rotated(x, c, s):
    a, b = x.float().chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_append(s):
    start, lens, Q = s["start"].long(), s["lens"].long(), s["max_q"]
    T, B, dev, blk = s["q"].shape[0], lens.numel(), s["q"].device, s["block"]
    pages, Hkv, P, D = s["k"].shape
    news = start[1:] - start[:-1]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(start, t, right=True) - 1
    pos = lens[b] - news[b] + t - start[b]                                 # a token's place in its cache
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _rotated(s["q"], cos, sin).to(torch.bfloat16)
    # the blocks that get new tokens, a padded list for each sequence
    before = lens - news
    n = (Q + blk - 2) // blk + 1
    first = before // blk
    index = first[:, None] + torch.arange(n, device=dev)                   # [B, n]
    live = index * blk < lens[:, None]
    page = s["table"].gather(1, (index * blk // P).clamp(max=s["table"].shape[1] - 1)).long()
    slot = index % (P // blk)
    cell = index[..., None] * blk + torch.arange(blk, device=dev)          # [B, n, blk]
    is_new = (cell >= before[:, None, None]) & (cell < lens[:, None, None])
    is_old = cell < before[:, None, None]
    token = (start[:-1, None, None] + cell - before[:, None, None]).clamp(0, T - 1)
    pg, sl = page[live], slot[live]
    new_m, old_m = is_new[live][:, None, :, None], is_old[live][:, None, :, None]
    for codes, scale, x in ((s["k"], s["k_scale"], _rotated(s["new_k"], cos, sin)),
                            (s["v"], s["v_scale"], s["new_v"].float())):
        view = codes.view(torch.float8_e4m3fn).view(pages, Hkv, P // blk, blk, D)
        had, s0 = view[pg, :, sl].float(), scale[pg, :, sl]                # [M, Hkv, blk, D], [M, Hkv]
        fresh = x[token[live]].permute(0, 2, 1, 3)                         # [M, Hkv, blk, D]
        big = torch.where(new_m & torch.isfinite(fresh), fresh.abs(), 0.0).amax((-1, -2))
        m, e = torch.frexp(big)                                            # big = m * 2^e, m in [1/2, 1)
        e = torch.where(big == 0, MIN_SCALE_EXP, torch.where(m <= 0.875, e - 9, e - 8))
        want = torch.ldexp(torch.ones_like(big), e.clamp(min=MIN_SCALE_EXP))
        s1 = torch.where(old_m.any(2)[..., 0], torch.maximum(s0, want), want)
        inv = (1.0 / s1)[..., None, None]
        put = torch.where(new_m, fresh * inv, had * s0[..., None, None] * inv)
        put = put.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        keep = view.view(torch.uint8)[pg, :, sl]
        grown = old_m & (s1 != s0)[..., None, None]
        codes.view(pages, Hkv, P // blk, blk, D)[pg, :, sl] = torch.where(new_m | grown, put, keep)
        scale[pg, :, sl] = s1
    return _appended(s, q)


def _plain_verify(s):
    drafts, target, guess = s["drafts"].long(), s["target"], s["guess"]
    B, S = drafts.shape
    V, dev = target.shape[-1], target.device
    p = target[:, :S].gather(-1, drafts[..., None])[..., 0].float()
    g = torch.ones_like(p) if guess is None else guess.gather(-1, drafts[..., None])[..., 0].float()
    # products of two fp32 numbers are exact in 64 bits
    ok = s["u"].double() * g.double() < p.double()
    count = torch.cumprod(ok.int(), -1).sum(-1)                            # [B]
    rows = torch.arange(B, device=dev)
    unit = float(1 << WEIGHT_BITS)

    def whole(x):        # probabilities as integers: their sums do not depend on the order
        return torch.round(x.float().clamp(0, 1) * unit).long()

    P = whole(target[rows, count])
    at = count.clamp(max=S - 1)
    x = drafts[rows, at]
    G = torch.zeros_like(P).scatter_(1, x[:, None], 1 << WEIGHT_BITS) if guess is None \
        else whole(guess[rows, at])
    W = torch.where((count < S)[:, None], (P - G).clamp(min=0), P)
    W = torch.where((W.sum(-1) == 0)[:, None], P, W)
    c = torch.cumsum(W, -1)
    total = c[:, -1]
    r = torch.floor(s["u_next"] * 2.0 ** 24).long().clamp(0, (1 << 24) - 1)
    mark = (total >> 24) * r + (((total & ((1 << 24) - 1)) * r) >> 24)     # floor(total * r / 2^24)
    nxt = (c > mark[:, None]).int().argmax(-1)
    nxt = torch.where(total == 0, -1, nxt)
    i = torch.arange(S + 1, device=dev)
    padded = torch.cat([drafts, torch.zeros_like(drafts[:, :1])], 1)
    tokens = torch.where(i < count[:, None], padded, torch.where(i == count[:, None], nxt[:, None], -1))
    return {"tokens": tokens.int(), "count": count.int()}


# ------------------------------------------------------------------ cost and 64-bit values

def work(case):
    if case["op"] == "verify":
        B, S, V = case["batch"], case["drafts"], case["vocab"]
        size = 4 if case["kind"] == "fp32" else 2
        # one target row of each sequence; the draft's row too where a draft is rejected (about
        # one in seven is, with these inputs)
        rejected = 1 - 0.85 ** S if case["draft_probs"] else 0.0
        return {"bytes": B * V * size * (1 + rejected) + B * S * (size * 2 + 8),
                "flops": 2 * B * V * (1 + rejected)}
    B, q, Hq, Hkv, D = case["batch"], case["q"], case["heads"], case["kv_heads"], case["dim"]
    share = 0.75 if case["ragged"] else 1.0       # mean over the ragged lengths
    T = max(1.0, B * q * share) if q > 1 else B
    if case["op"] == "attn":
        N = B * max(1.0, case["length"] * share)
        return {"bytes": 2 * N * Hkv * (D + 4 / case["block"]) + 4 * T * Hq * D,
                "flops": 4 * (N / B) * T * Hq * D}
    return {"bytes": T * (4 * Hq * D + 6 * Hkv * D + 4 * D + 8 * Hkv / case["block"]),
            "flops": 3 * T * (Hq + Hkv) * D + 4 * T * Hkv * D}


def exact(case, seed):
    if case["op"] == "verify":
        return None                       # whole numbers only
    s = prepare(case, seed)
    start, lens = s["start"].tolist(), s["lens"].tolist()
    pages, Hkv, P, D = s["k"].shape
    T, Hq, _ = s["q"].shape
    if case["op"] == "append":
        # the rotated queries; the stored codes are roundings that have no 64-bit value
        out = torch.empty(T, Hq, D, dtype=torch.float64, device=s["q"].device)
        half = D // 2
        for b, n in enumerate(lens):
            i0, i1 = start[b], start[b + 1]
            c = s["cos"][n - (i1 - i0):n].double()[:, None]
            sn = s["sin"][n - (i1 - i0):n].double()[:, None]
            x = s["q"][i0:i1].double()
            out[i0:i1, :, :half] = x[..., :half] * c - x[..., half:] * sn
            out[i0:i1, :, half:] = x[..., half:] * c + x[..., :half] * sn
        return {"q": out, "k": None, "v": None, "k_scale": None, "v_scale": None}
    out = torch.empty(T, Hq, D, dtype=torch.float64, device=s["q"].device)
    group = Hq // Hkv
    for b, n in enumerate(lens):
        ids = s["table"][b, :-(-n // P)].long()

        def rows(codes, scale):
            x = codes[ids].view(torch.float8_e4m3fn).double()
            x = x * scale[ids].double().repeat_interleave(case["block"], -1)[..., None]
            return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :n]

        k, v = rows(s["k"], s["k_scale"]), rows(s["v"], s["v_scale"])
        i0, i1 = start[b], start[b + 1]
        for i in range(i0, i1):
            m = n - (i1 - 1 - i)          # tokens that this one sees
            x = s["q"][i].double().view(Hkv, group, D) / math.sqrt(D)
            z = torch.softmax(torch.matmul(x, k[:, :m].transpose(1, 2)), -1)
            out[i] = torch.matmul(z, v[:, :m]).view(Hq, D)
    return out
