"""Inputs and plain 64-bit references of the cached-attention tests (CPU, loops)."""
import math

import numpy as np
import torch

import weight_streaming_skinny_gb300 as dl

F8 = torch.float8_e4m3fn


class Step:
    """One call's sequences over a paged cache, on the CPU: `lens` cached tokens (the new ones
    included) and `news` new tokens of each sequence."""

    def __init__(self, lens, news, *, heads=8, kv_heads=2, dim=128, page=16, block=16, seed=0,
                 spare_pages=2, extra_cols=1, code_std=1.0, pow2=True):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens, self.news = g, list(lens), list(news)
        self.heads, self.kv_heads, self.dim, self.page, self.block = heads, kv_heads, dim, page, block
        self.B, self.T, self.max_q = len(self.lens), sum(self.news), max(list(self.news) + [0])
        need = [-(-max(n, 0) // page) for n in self.lens]
        self.cols = max(need + [0]) + extra_cols
        self.pages = sum(need) + spare_pages
        order = torch.randperm(self.pages, generator=g)
        self.table = torch.full((self.B, self.cols), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m].int()
            at += m
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(self.news)]), dtype=torch.int32)
        shape = (self.pages, kv_heads, page, dim)
        self.k, self.v = ((code_std * 60 * torch.randn(shape, generator=g)).clamp(-448, 448).to(F8)
                          for _ in range(2))
        s = torch.randn(2, self.pages, kv_heads, page // block, generator=g)
        s = torch.exp2(torch.round(s) - 6) if pow2 else torch.exp(s * 0.7 - 4.2)
        self.k_scale, self.v_scale = s[0].contiguous(), s[1].contiguous()
        self.q, self.new_k, self.new_v = (torch.randn(self.T, h, dim, generator=g).bfloat16()
                                          for h in (heads, kv_heads, kv_heads))

    def cache(self, dev):
        c = dl.PagedKVCache(self.k.to(dev), self.v.to(dev), self.k_scale.to(dev), self.v_scale.to(dev))
        return c

    def seqs(self, dev):
        return (self.table.to(dev), torch.tensor(self.lens, dtype=torch.int32, device=dev),
                self.start.to(dev))

    def slots(self, b, n):
        """(page, offset) of the first n tokens of sequence b."""
        return [(int(self.table[b, j // self.page]), j % self.page) for j in range(n)]


def dequantised(step, codes, scale):
    return codes.double() * scale.double().repeat_interleave(step.block, -1)[..., None]


def reference(step, scale=None):
    """(out, lse, spread, biggest): attention in 64 bits; spread = sum_j p_j |V_j| and biggest =
    max_j |V_j| over the seen tokens, for error bounds.  Tokens of a page outside the pool are
    not seen."""
    scale = step.dim ** -0.5 if scale is None else scale
    K, V = (dequantised(step, c, s) for c, s in ((step.k, step.k_scale), (step.v, step.v_scale)))
    G = step.heads // step.kv_heads
    out = torch.zeros(step.T, step.heads, step.dim, dtype=torch.float64)
    spread, biggest = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((step.T, step.heads), -math.inf, dtype=torch.float64)
    for b in range(step.B):
        for i in range(step.news[b]):
            t = int(step.start[b]) + i
            seen = min(step.lens[b] - step.news[b] + i + 1, step.cols * step.page)
            at = [(p, o) for p, o in step.slots(b, max(seen, 0)) if 0 <= p < step.pages]
            if not at:
                continue
            pg, of = (torch.tensor(x) for x in zip(*at))
            for h in range(step.heads):
                k, v = K[pg, h // G, of], V[pg, h // G, of]
                s = (k @ step.q[t, h].double()) * scale
                p = torch.softmax(s, 0)
                out[t, h] = p @ v
                spread[t, h] = p @ v.abs()
                biggest[t, h] = v.abs().amax(0)
                lse[t, h] = torch.logsumexp(s, 0)
    return out, lse, spread, biggest


def bound(step, out, spread, biggest):
    """Largest error of one output element.  The bf16 rounding is at most 2^-9 of a binade's top:
    2^-8 |out|.  A probability is multiplied as the sum of two e4m3 parts: relative error at most
    2^-8, or an absolute one below 2^-22 of the row's largest weighted probability for each of the
    tokens; a relative 2^-8 covers an fp16 or fp32 probability too.  Scores are exact to about
    2^-16 of the row's largest, allowed 2^-10 relative in p; all of it in |V|."""
    n = max(step.lens + [1])
    return 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -10) * spread + n * 2.0 ** -22 * biggest + 1e-30


def e4m3_nearest(x):
    """Codes of fp64 numpy values in [-448, 448], to nearest even, from the format's definition."""
    mags = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127])
    a = np.abs(x)
    hi = np.clip(np.searchsorted(mags, a), 1, 126)
    lo = hi - 1
    d_lo, d_hi = a - mags[lo], mags[hi] - a
    idx = np.where(d_lo < d_hi, lo, np.where(d_hi < d_lo, hi, np.where(lo % 2 == 0, lo, hi)))
    idx = np.where(a == 0, 0, idx)
    return (idx | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def reference_append(step, cos=None, sin=None, positions=None):
    """(q_out fp32 before rounding, k, v codes uint8, k_scale, v_scale) after the append: loops in
    fp32 with separate roundings, codes from the format's definition."""
    f = np.float32
    rot = 0 if cos is None else 2 * cos.shape[1]

    def rotate(x, pos):
        y = x.astype(f).copy()
        if rot:
            h = rot // 2
            c, s = cos[pos], sin[pos]
            a, b = x[..., :h].astype(f), x[..., h:rot].astype(f)
            y[..., :h] = (a * c).astype(f) - (b * s).astype(f)
            y[..., h:rot] = (b * c).astype(f) + (a * s).astype(f)
        return y

    q = step.q.float().numpy().copy()
    codes = {n: getattr(step, n).view(torch.uint8).numpy().copy() for n in ("k", "v")}
    scales = {n: getattr(step, n + "_scale").numpy().copy() for n in ("k", "v")}
    value = np.array([float(torch.tensor([c], dtype=torch.uint8).view(F8)[0]) for c in range(256)], dtype=f)
    for b in range(step.B):
        n, L = step.news[b], min(step.lens[b], step.cols * step.page)
        fresh = {}
        for i in range(n):
            t, idx = int(step.start[b]) + i, L - n + i
            pos = idx if positions is None else int(positions[t])
            pos = min(max(pos, 0), (len(cos) if rot else 1) - 1)
            q[t] = rotate(q[t], pos)
            if idx >= 0:
                fresh.setdefault(idx // step.block, []).append(
                    (idx % step.block, rotate(step.new_k[t].float().numpy(), pos), step.new_v[t].float().numpy()))
        for blk, rows in fresh.items():
            at = blk * step.block
            pg = int(step.table[b, at // step.page])
            if not 0 <= pg < step.pages:
                continue
            c, o = (at % step.page) // step.block, at % step.page
            held = rows[0][0]                       # tokens already in the block
            for name, col in (("k", 1), ("v", 2)):
                for h in range(step.kv_heads):
                    x = np.stack([r[col][h] for r in rows])
                    fin = np.abs(x[np.isfinite(x)])
                    amax = float(fin.max()) if fin.size else 0.0
                    e = -40
                    while 448.0 * 2.0 ** e < amax:
                        e += 1
                    s0, s1 = scales[name][pg, h, c], f(2.0 ** e)
                    if held and not s0 < s1:
                        s1 = s0
                    inv = f(1) / s1
                    if held and s1 != s0:
                        old = codes[name][pg, h, o:o + held]
                        y = ((value[old] * s0).astype(f) * inv).astype(f)
                        new = e4m3_nearest(np.clip(y, -448, 448).astype(np.float64))
                        codes[name][pg, h, o:o + held] = np.where(np.isnan(y), 127, new)
                    with np.errstate(invalid="ignore"):
                        y = (x * inv).astype(f)
                        new = e4m3_nearest(np.nan_to_num(np.clip(y, -448, 448)).astype(np.float64))
                    codes[name][pg, h, o + held:o + held + len(rows)] = np.where(np.isnan(y), 127, new)
                    scales[name][pg, h, c] = s1
    return q, codes["k"], codes["v"], scales["k"], scales["v"]


def same_codes(a, b):
    """Equal codes; any two NaN codes are equal."""
    a, b = np.asarray(a), np.asarray(b)
    return np.array_equal(np.where(a & 127 == 127, 127, a), np.where(b & 127 == 127, 127, b))


def rope_tables(positions, rotary_dim, base=10000.0):
    a = np.outer(np.arange(positions), base ** (-np.arange(0, rotary_dim, 2) / rotary_dim))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def reference_verify(drafts, target, guess, u, u_next, lens=None):
    """(tokens, count) with whole Python numbers: probabilities as multiples of 2^-44."""
    B, S = drafts.shape
    V = target.shape[2]
    tokens = np.full((B, S + 1), -1, np.int32)
    count = np.zeros(B, np.int32)

    def whole(row):
        y = np.clip(np.nan_to_num(np.asarray(row, np.float64), nan=0.0), 0, 1) * 2.0 ** 44
        return [int(v) for v in np.rint(y)]

    for b in range(B):
        n = S if lens is None else int(lens[b])
        c = 0
        while c < n:
            x = int(drafts[b, c])
            if not 0 <= x < V:
                break
            g = 1.0 if guess is None else float(guess[b, c, x])
            if not float(u[b, c]) * g < float(target[b, c, x]):
                break
            c += 1
        P = whole(target[b, c])
        W = P
        if c < n:
            x = int(drafts[b, c])
            G = whole(guess[b, c]) if guess is not None else [(1 << 44) if v == x else 0 for v in range(V)]
            W = [max(p - g, 0) for p, g in zip(P, G)]
            if sum(W) == 0:
                W = P
        total = sum(W)
        nxt = -1
        if total:
            mark = total * min(int(float(u_next[b]) * 2 ** 24), 2 ** 24 - 1) >> 24
            run = 0
            for v, w in enumerate(W):
                run += w
                if run > mark:
                    nxt = v
                    break
        tokens[b, :c] = drafts[b, :c]
        tokens[b, c] = nxt
        count[b] = c
    return tokens, count
