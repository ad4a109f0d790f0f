"""Plain 64-bit references of block_norm, linear_adapters and the pages of the cache (CPU), with the error
bounds that their tests use."""
import torch

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64

# A rounding to a type is off by at most half a step, relative to the value.
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def norm64(v, kind, w, b, eps, offset):
    """(N(v), bound of its error if v is exact): v fp64 [rows, dim].

    The sums run over at most 64 terms a thread (a fused multiply-add each), then 10 levels of a tree:
    74 roundings of 2^-24, less than 2^-17 of a sum of squares and 2^-18 of its root; the products
    after it add 8 more.  Together below 2^-17 of |c / sqrt(..)  (offset + w)|, and 2^-23 of the bias' sum.  A
    centred value is off by the rounding of two subtractions of the mean, 2^-23 of max |v|, and the
    mean's own error is taken off by the second pass: 2^-22 max |v| covers both.
    """
    if kind is None:
        return v, torch.zeros_like(v)
    off = torch.zeros_like(v[:, :1])
    if kind == "layer":
        off = 2.0 ** -22 * v.abs().amax(-1, keepdim=True)
        v = v - v.mean(-1, keepdim=True)
    inv = 1 / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
    scale = torch.ones_like(v) if w is None else (offset + w.double()).expand_as(v)
    y = v * inv * scale
    # a centred value's error reaches the others through the root: its part of the mean square is at most itself
    err = 2.0 ** -17 * y.abs() + 2 * off * inv * scale.abs()
    if b is not None:
        y = y + b.double()
        err = err + 2.0 ** -23 * (y.abs() + b.double().abs())
    return y, err


def block_norm64(y, h, post, pre, gate, act, scale, h_scale):
    """((r, x), (bounds before the rounding to the outputs' types)).  post, pre: None or (kind, w, b, eps,
    offset); gate fp64-castable, broadcast to [rows, dim]."""
    like = y if y is not None else h
    r, dr = torch.zeros(like.shape, dtype=F64), torch.zeros(like.shape, dtype=F64)
    if y is not None:
        u, du = norm64(y.double(), *(post or (None,) * 5))
        if gate is not None:
            g = gate.double().expand(like.shape)
            if act:
                g = torch.sigmoid(g)
            # the gate: expf to 2 units of 2^-23, a sum and a quotient
            u, du = u * g, (du + 2.0 ** -20 * u.abs()) * g.abs()
        r, dr = scale * u, abs(scale) * du + 2.0 ** -23 * (scale * u).abs()
    if h is not None:
        r = r + h_scale * h.double()
        dr = dr + 2.0 ** -23 * ((h_scale * h.double()).abs() + r.abs())
    if pre is None:
        return (r, r), (dr, dr)
    x, dx = norm64(r, *pre)
    kind, w, b, eps, offset = pre
    c = r - r.mean(-1, keepdim=True) if kind == "layer" else r
    dc = dr + (dr.mean(-1, keepdim=True) if kind == "layer" else 0)
    inv = 1 / torch.sqrt(c.square().mean(-1, keepdim=True) + eps)
    s = torch.ones_like(r) if w is None else (offset + w.double()).abs().expand_as(r)
    # d(c inv) = inv dc - c inv^3 mean(c dc), to the second order doubled
    dx = dx + 2 * s * (inv * dc + c.abs() * inv ** 3 * (c.abs() * dc).mean(-1, keepdim=True))
    return (r, x), (dr, dx)


def assert_near(got, want, bound, what=""):
    """|got - want| <= bound + the rounding to got's type (below its normal range 2^-126: a step of 2^-133
    in bf16, 2^-149 in fp32)."""
    g = got.detach().cpu().double()
    tiny = 2.0 ** -134 if got.dtype == BF16 else 2.0 ** -150
    limit = bound * (1 + HALF[got.dtype]) + HALF[got.dtype] * want.abs() + tiny
    bad = ~((g - want).abs() <= limit)
    bad &= ~(torch.isnan(g) & torch.isnan(want)) & ~(g == want)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first {i}: got "
                             f"{float(g[tuple(i)])!r}, want {float(want[tuple(i)])!r} +- {float(limit[tuple(i)])!r}")


def adapters64(x, a, b, index, scale, ranks, cols, base, whole):
    """(out fp64 [T, N], bound of its error before rounding); `whole`: first products go whole into the second.

    A product of two bf16 is exact in fp32.  A tensor-core sum of 16 products rounds, or cuts, to fp32 at
    each step: K / 16 + 32 sums (the joins among them) of at most 2^-23 of sum |a x| each.  Then the
    scale (2^-24), the split into parts (2^-18, or 2^-26 of three parts), and the sums over r likewise, of
    2^-23 sum |low b| for each of the up to 3 r / 16 + 8.
    """
    T, (num, N, R) = x.shape[0], b.shape
    out = torch.zeros(T, N, dtype=F64) if base is None else base.double().clone()
    err = 2.0 ** -24 * out.abs()
    K = x.shape[1]
    for t in range(T):
        i = int(index[t])
        if not 0 <= i < num:
            continue
        r = R if ranks is None else min(max(int(ranks[i]), 0), R)
        s = 1.0 if scale is None else float(scale[i])
        n0 = 0
        for p, c in enumerate(cols):
            A, B = a[i, p * R:p * R + r].double(), b[i, n0:n0 + c, :r].double()
            low, spread = s * (A @ x[t].double()), abs(s) * (A.abs() @ x[t].double().abs())
            dlow = (K / 16 + 32) * 2.0 ** -23 * spread + (2.0 ** -23 + (2.0 ** -26 if whole else 2.0 ** -18)) * low.abs()
            out[t, n0:n0 + c] += B @ low
            err[t, n0:n0 + c] += B.abs() @ dlow + (3 * r / 16 + 8) * 2.0 ** -23 * (B.abs() @ low.abs())
            n0 += c
    return out, err + 2.0 ** -24 * out.abs()


class Pool:
    """The state of a PagePool in Python lists; steps give the copies (from, to, tokens) that they make."""

    def __init__(self, num_pages, page, rows, cols):
        self.page, self.cols = page, cols
        self.refs, self.lens = [0] * num_pages, [0] * rows
        self.table = [[-1] * cols for _ in range(rows)]

    def length(self, row):
        return min(max(self.lens[row], 0), self.cols * self.page)

    def pages(self, row):
        return -(-self.length(row) // self.page)

    def inside(self, p):
        return 0 <= p < len(self.refs)

    def take(self, n):
        free = [p for p, c in enumerate(self.refs) if c <= 0]
        return free[:n]

    def free(self, rows):
        for r in rows:
            if not 0 <= r < len(self.lens):
                continue
            for p in self.table[r][:self.pages(r)]:
                if self.inside(p) and self.refs[p] > 0:
                    self.refs[p] -= 1
            self.lens[r] = 0

    def _served(self, wants):
        """wants: None (refused) or pages asked for, of each item; pages for each served item, else None."""
        free = self.take(len(self.refs))
        out, asked = [], 0
        for w in wants:
            if w is None:
                out.append(None)
                continue
            asked += w
            out.append(free[asked - w:asked] if w == 0 or asked <= len(free) else None)
        return out

    def reserve(self, rows, tokens):
        wants, seen = [], set()
        for r, n in zip(rows, tokens):
            ok = 0 <= r < len(self.lens) and r not in seen and n >= 0 and \
                self.length(r) + n <= self.cols * self.page
            seen.add(r)
            wants.append(-(-(self.length(r) + n) // self.page) - self.pages(r) if ok else None)
        got = self._served(wants)
        for r, n, pages in zip(rows, tokens, got):
            if pages is not None:
                first = self.pages(r)
                for i, p in enumerate(pages):
                    self.table[r][first + i] = p
                    self.refs[p] = 1
                self.lens[r] = self.length(r) + n
        return [int(g is not None) for g in got]

    def fork(self, parents, children):
        wants, seen, lens = [], set(), [self.length(r) for r in range(len(self.lens))]
        inside = lambda r: 0 <= r < len(self.lens)   # noqa: E731
        for f, c in zip(parents, children):
            ok = inside(f) and inside(c) and f != c and c not in seen and self.lens[c] <= 0
            seen.add(c)
            wants.append(int(lens[f] % self.page > 0) if ok else None)
        got = self._served(wants)
        served = [(f, c, lens[f], pages) for f, c, pages in zip(parents, children, got) if pages is not None]
        copies = []
        for f, c, n, pages in served:           # new pages first, then the shared ones' counts
            self.lens[c] = n
            full, tail = n // self.page, n % self.page
            if tail:
                p, q = self.table[f][full], pages[0]
                self.table[c][full] = q
                self.refs[q] = 1
                if self.inside(p):
                    copies.append((p, q, tail))
        for f, c, n, _ in served:
            for i in range(n // self.page):
                p = self.table[c][i] = self.table[f][i]
                if self.inside(p):
                    self.refs[p] += 1
        return [int(g is not None) for g in got], copies

    def compact(self):
        live = sum(c > 0 for c in self.refs)
        src = [p for p, c in enumerate(self.refs) if c > 0 and p >= live]
        dst = [p for p, c in enumerate(self.refs) if c <= 0 and p < live]
        to = dict(zip(src, dst))
        for r in range(len(self.lens)):
            for i in range(self.pages(r)):
                self.table[r][i] = to.get(self.table[r][i], self.table[r][i])
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        return live, list(to.items())
