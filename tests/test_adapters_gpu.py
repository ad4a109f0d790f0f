"""linear_adapters against its formula in 64 bits, element by element."""
import itertools

import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from step_util import BF16, F32, adapters64, assert_near

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, T, K, N, R, num, *, cols=None, base="bf16", f32=False, ranks=True, scale=True, order="mixed", seed=0,
                 none=0.1):
        g = torch.Generator().manual_seed(seed)
        self.T, self.K, self.N, self.cols, self.f32 = T, K, N, cols or [N], f32
        randn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
        self.x = randn(T, K).to(BF16)
        self.a = (randn(num, len(self.cols) * R, K) * K ** -0.5).to(BF16)
        self.b = (randn(num, N, R) * R ** -0.5).to(BF16)
        self.base = None if base is None else randn(T, N).to({"bf16": BF16, "fp32": F32}[base])
        self.scale = torch.rand(num, generator=g) + 0.5 if scale else None
        self.ranks = None
        if ranks:
            self.ranks = torch.randint(0, R + 1, (num,), generator=g).int()
            for i in range(num):            # what lies past an adapter's rank reaches nothing
                r = int(self.ranks[i])
                self.a.view(num, len(self.cols), R, K)[i, :, r:] = float("nan")
                self.b[i, :, r:] = float("nan")
        self.index = torch.randint(0, num, (T,), generator=g).int()
        if order == "runs":
            self.index = self.index.sort()[0]
        if none:
            lost = torch.rand(T, generator=g) < none
            self.index[lost] = torch.tensor([-1, num, 2 ** 31 - 1, -2 ** 31]).int()[torch.arange(int(lost.sum())) % 4]

    def adapters(self, dev):
        on = lambda t: None if t is None else t.to(dev)   # noqa: E731
        return dl.Adapters(on(self.a), on(self.b), scale=on(self.scale), ranks=on(self.ranks), parts=self.cols)

    def run(self, dev, **kw):
        on = lambda t: None if t is None else t.to(dev)   # noqa: E731
        if self.f32 and "out_f32" not in kw:
            kw["out_f32"] = torch.empty(self.T, self.N, device=dev)
        out = dl.linear_adapters(on(self.x), self.adapters(dev), on(self.index), on(self.base), **kw)
        return out, kw.get("out_f32")

    def check(self, out, out32=None):
        want, bound = adapters64(self.x, self.a, self.b, self.index, self.scale, self.ranks, self.cols, self.base,
                                 out32 is not None)
        assert_near(out, want, bound, "out")
        if out32 is not None:
            assert_near(out32, want, bound, "out_f32")
            assert torch.equal(out, out32.to(BF16))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 33, 64, 255, 256, 257, 300, 700])
def test_token_counts(cuda_device, T):
    for order, num in (("mixed", 3), ("runs", 5), ("mixed", 200)):
        c = Case(T, 136, 50, 16, num, order=order, seed=T)
        c.check(*c.run(cuda_device))


@pytest.mark.parametrize("K", [8, 16, 24, 32, 40, 64, 120, 264, 1000, 4096, 8200])
@pytest.mark.parametrize("T", [1, 5, 20, 300])
def test_depths(cuda_device, K, T):
    c = Case(T, K, 40, 8, 4, seed=K)
    c.check(*c.run(cuda_device))


@pytest.mark.parametrize("N", [1, 2, 3, 4, 7, 15, 16, 17, 33, 63, 64, 65, 127, 129, 200, 1001])
def test_widths(cuda_device, N):
    for T, base in ((1, "bf16"), (18, "fp32"), (300, None)):
        c = Case(T, 64, N, 16, 4, base=base, seed=N)
        c.check(*c.run(cuda_device))


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 96, 128, 256])
@pytest.mark.parametrize("f32", [False, True])
def test_ranks(cuda_device, R, f32):
    for T, ranks in ((1, False), (19, True), (290, True)):
        c = Case(T, 128, 72, R, 6, ranks=ranks, f32=f32, seed=R)
        c.check(*c.run(cuda_device))


@pytest.mark.parametrize("cols", [[16, 16], [32, 16, 17], [16] * 7 + [5], [160, 32, 32], [96, 100]])
def test_parts(cuda_device, cols):
    for T in (1, 16, 40, 280):
        c = Case(T, 104, sum(cols), 24, 5, cols=cols, seed=len(cols))
        c.check(*c.run(cuda_device))


@pytest.mark.parametrize("base,f32,scale,ranks", list(itertools.product(["bf16", "fp32", None], [False, True], [False, True],
                                                                   [False, True])))
def test_forms(cuda_device, base, f32, scale, ranks):
    for T in (3, 270):
        c = Case(T, 96, 48, 16, 4, base=base, f32=f32, scale=scale, ranks=ranks)
        c.check(*c.run(cuda_device))


@pytest.mark.parametrize("T", [1, 4, 260])
def test_without_adapters(cuda_device, T):
    """No token has one: out is base, bit for bit, or zeros."""
    c = Case(T, 64, 80, 16, 4, none=1.1)
    out, _ = c.run(cuda_device)
    assert torch.equal(out.cpu(), c.base)
    c.base = None
    assert not c.run(cuda_device)[0].any()


@pytest.mark.parametrize("T", [2, 16, 300])
def test_in_place(cuda_device, T):
    """out is base: rows without an adapter are not written (a NaN's payload stays)."""
    c = Case(T, 64, 80, 16, 4, none=0.5)
    c.index[0] = -1
    want, _ = c.run(cuda_device)
    base = c.base.to(cuda_device)
    base.view(torch.int16)[0] = 0x7fab
    out = dl.linear_adapters(c.x.to(cuda_device), c.adapters(cuda_device), c.index.to(cuda_device), base, out=base)
    assert out is base and bool((base.view(torch.int16)[0] == 0x7fab).all())
    assert torch.equal(out[1:], want[1:])
    c = Case(T, 64, 80, 16, 4, base="fp32", f32=True)
    want = c.run(cuda_device)
    base = c.base.to(cuda_device)
    out, _ = c.run(cuda_device, out_f32=base)
    out2 = dl.linear_adapters(c.x.to(cuda_device), c.adapters(cuda_device), c.index.to(cuda_device), c.base.to(cuda_device),
                              out_f32=torch.empty_like(base))
    assert torch.equal(out, want[0]) and torch.equal(out2, want[0])
    base = c.base.to(cuda_device)
    dl.linear_adapters(c.x.to(cuda_device), c.adapters(cuda_device), c.index.to(cuda_device), base, out_f32=base)
    assert torch.equal(base, want[1])


@pytest.mark.parametrize("T", [5, 300])
def test_views(cuda_device, T):
    """Rows of wider tensors, aligned for wide accesses and not; what lies beside them stays."""
    for off, N in ((0, 96), (1, 95), (2, 94), (4, 92), (8, 64)):
        c = Case(T, 64, N, 16, 4, f32=True, seed=off)
        pad = lambda t, n: torch.nn.functional.pad(t.to(cuda_device), (n, 8))   # noqa: E731
        x, base = pad(c.x, 8)[:, 8:72], pad(c.base, off)[:, off:off + N]
        out, out32 = (torch.full((T, N + off + 9), 7.0, dtype=d, device=cuda_device) for d in (BF16, F32))
        v, v32 = out[:, off:off + N], out32[:, off:off + N]
        dl.linear_adapters(x, c.adapters(cuda_device), c.index.to(cuda_device), base, out=v, out_f32=v32)
        c.check(v, v32)
        for t in (out, out32):
            assert bool((t[:, :off] == 7).all()) and bool((t[:, off + N:] == 7).all())


def test_a_projection_of_several(cuda_device):
    """Parts are what separate calls on the columns give, bit for bit."""
    for T in (1, 16, 300):
        c = Case(T, 256, 128, 16, 4, cols=[64, 32, 32])
        out, _ = c.run(cuda_device)
        got, n0 = torch.empty_like(out), 0
        for p, n in enumerate(c.cols):
            one = dl.Adapters(c.a[:, 16 * p:16 * p + 16].contiguous().to(cuda_device), c.b[:, n0:n0 + n].contiguous().to(cuda_device),
                              scale=c.scale.to(cuda_device), ranks=c.ranks.to(cuda_device))
            dl.linear_adapters(c.x.to(cuda_device), one, c.index.to(cuda_device), c.base.to(cuda_device)[:, n0:n0 + n],
                               out=got[:, n0:n0 + n])
            n0 += n
        assert torch.equal(got, out)


@pytest.mark.parametrize("T", [16, 256, 600])
def test_tokens_keep_to_themselves(cuda_device, T):
    """A token's result is the same bit for bit in any company and order; NaN and infinities of one
    token's input, or of another adapter, do not reach it."""
    c = Case(T, 512, 96, 16, 5, ranks=False, none=0.0, f32=True, seed=T)
    out, out32 = c.run(cuda_device)
    p = torch.randperm(T, generator=torch.Generator().manual_seed(1))
    d = Case(T, 512, 96, 16, 5, ranks=False, none=0.0, f32=True, seed=T)
    d.x, d.index, d.base = c.x[p], c.index[p], c.base[p]
    got, got32 = d.run(cuda_device)
    assert torch.equal(got.cpu(), out.cpu()[p]) and torch.equal(got32.cpu(), out32.cpu()[p])
    d.a[2], d.b[3, 5], d.x[1] = float("nan"), float("inf"), float("inf")
    bad, _ = d.run(cuda_device)
    keep = (d.index != 2) & (d.index != 3)
    keep[1] = False
    assert torch.equal(bad.cpu()[keep], out.cpu()[p][keep])
    assert bool(torch.isnan(bad.cpu()[(d.index == 2)].float()).all())


def test_infinite_weights(cuda_device):
    """An infinity in b times a value that its first part holds whole is an infinity, not NaN."""
    for T in (1, 300):
        c = Case(T, 64, 32, 8, 2, ranks=False, none=0.0, base=None, scale=False)
        c.x[:], c.a[:], c.b[:] = 1.0, 0.0, 0.25
        c.a[:, 0, 0] = 1.5                  # first products: 1.5, then zeros
        c.b[:, 4, 0], c.b[:, 5, 0], c.b[:, 6, 1] = float("inf"), -float("inf"), float("inf")
        out, _ = c.run(cuda_device)
        o = out.cpu().float()
        assert bool((o[:, 4] == float("inf")).all()) and bool((o[:, 5] == -float("inf")).all())
        assert bool(torch.isnan(o[:, 6]).all()) and bool((o[:, :4] == 0.375).all())
        c.a[:, 0, 0] = 3e38                 # beyond what the first part can round to
        c.b[:] = 2.0 ** -100
        out, _ = c.run(cuda_device)
        assert bool(torch.isfinite(out).all()) and bool((out > 0).all())


def test_large_store(cuda_device):
    """Offsets beyond 2^31 bytes and elements in the store."""
    num, R, K, N = 5000, 64, 8192, 16
    a = torch.zeros(num, R, K, dtype=BF16, device=cuda_device)
    b = torch.zeros(num, N, R, dtype=BF16, device=cuda_device)
    a[-1, 0, -1], b[-1, :, 0] = 2.0, 3.0
    x = torch.ones(3, K, dtype=BF16, device=cuda_device)
    index = torch.tensor([num - 1, 0, num - 1], dtype=torch.int32, device=cuda_device)
    out = dl.linear_adapters(x, dl.Adapters(a, b), index)
    assert out.tolist() == [[6.0] * N, [0.0] * N, [6.0] * N]


def test_many_adapters(cuda_device):
    """The largest store; a sort over all of them."""
    num = 16384
    c = Case(1000, 16, 16, 8, 8, none=0.0, ranks=False)
    a = torch.zeros(num, 8, 16, dtype=BF16, device=cuda_device)
    b = torch.zeros(num, 16, 8, dtype=BF16, device=cuda_device)
    at = torch.randperm(num, generator=torch.Generator().manual_seed(2))[:8]
    a[at], b[at] = c.a.to(cuda_device), c.b.to(cuda_device)
    want, _ = c.run(cuda_device)
    scale = torch.zeros(num, device=cuda_device)
    scale[at] = c.scale.to(cuda_device)
    got = dl.linear_adapters(c.x.to(cuda_device), dl.Adapters(a, b, scale=scale), at.int()[c.index.long()].to(cuda_device),
                             c.base.to(cuda_device))
    assert torch.equal(got, want)


def test_repeats_graphs_and_workspaces(cuda_device):
    """Bitwise repeatable on a workspace that holds anything past its zero prefix; two graphs on one
    workspace; the zero prefix stays; the linears go on with it."""
    for T in (16, 300):
        c = Case(T, 1024, 200, 16, 6, seed=T)
        ad, x, index, base = c.adapters(cuda_device), c.x.to(cuda_device), c.index.to(cuda_device), c.base.to(cuda_device)
        need = dl.adapters_workspace_bytes(T, ad)
        ws = dl.Workspace(need + 4096)
        want = dl.linear_adapters(x, ad, index, base)
        ws.tensor[dl.WORKSPACE_ZERO_BYTES:].fill_(0xff)
        assert torch.equal(dl.linear_adapters(x, ad, index, base, workspace=ws), want)
        assert not ws.tensor[:dl.WORKSPACE_ZERO_BYTES].any() and bool((ws.tensor[need:] == 0xff).all())
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(dl.linear_adapters(x, ad, index, base, workspace=ws))
            graphs.append(g)
        for g in graphs * 2:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        index.copy_(index.flip(0))
        for g in graphs:
            g.replay()
        again = dl.linear_adapters(x, ad, index, base, workspace=ws)
        assert all(torch.equal(o, again) for o in outs)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = dl.linear_adapters(x, ad, index, base, stream=side)
        side.synchronize()
        assert torch.equal(got, again)


def test_after_a_linear(cuda_device):
    """Beside linear_bf16: from its y, its y_f32, and into a view of a fused projection."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(16, 512, generator=g).to(BF16).to(cuda_device)
    w = (torch.randn(256, 512, generator=g) / 20).to(BF16).to(cuda_device)
    c = Case(16, 512, 256, 16, 4, cols=[128, 64, 64], base="fp32", f32=True)
    c.x = x.cpu()
    y32 = torch.empty(16, 256, device=cuda_device)
    y = dl.linear_bf16(x, w, out_f32=y32)
    torch.cuda.synchronize()
    c.base = y32.cpu()
    out32 = torch.empty_like(y32)
    ad, index = c.adapters(cuda_device), c.index.to(cuda_device)
    for _ in range(20):
        dl.linear_bf16(x, w, out=y, out_f32=y32)
        out = dl.linear_adapters(x, ad, index, y32, out_f32=out32)
    c.check(out, out32)


def test_refusals(cuda_device):
    c = Case(4, 64, 32, 16, 3)
    ad, x, index, base = c.adapters(cuda_device), c.x.to(cuda_device), c.index.to(cuda_device), c.base.to(cuda_device)
    for args, kw, match in (((x[:, :32], ad, index, base), {}, "x must"), ((x.float(), ad, index, base), {}, "x must"),
                            ((x, ad, index[:3], base), {}, "index"), ((x, ad, index.long(), base), {}, "index"),
                            ((x, ad, index, base[:, :16]), {}, "base"), ((x, ad, index, base.half()), {}, "base"),
                            ((x, ad, index, base), dict(out=base[:2]), "out"), ((x, ad, index, base), dict(out=base.float()), "out"),
                            ((x, ad, index, base), dict(out_f32=base), "out_f32"), ((x, ad, index.cpu(), base), {}, "index")):
        with pytest.raises(ValueError, match=match):
            dl.linear_adapters(*args, **kw)
    with pytest.raises(dl.DLError, match="workspace"):
        dl.linear_adapters(x, ad, index, base, workspace=dl.Workspace(1000))
    with pytest.raises(dl.DLError, match="overlap"):
        dl.linear_adapters(x, ad, index, base, out=x[:, :32])
    with pytest.raises(ValueError, match="add up"):
        dl.Adapters(ad.a, ad.b, parts=[16, 8])
    with pytest.raises(ValueError, match="scale"):
        dl.Adapters(ad.a, ad.b, scale=torch.ones(2, device=cuda_device))
    with pytest.raises(ValueError, match="b"):
        dl.Adapters(ad.a, ad.b.float())


@pytest.mark.parametrize("R", [8, 24, 64, 104, 128])
@pytest.mark.parametrize("base,f32", [("bf16", False), ("bf16", True), ("fp32", False), ("fp32", True), (None, False), (None, True)])
def test_long_runs(cuda_device, R, base, f32):
    """Runs of tokens of one adapter: whole tiles of 128, their ends, runs that are just too short; columns in
    whole blocks of 64, at a part's end and rows that allow no wide access; ranks that end inside 16."""
    g = torch.Generator().manual_seed(R)
    for N, cols, K in ((192, [128, 64], 72), (200, None, 1000), (100, None, 520), (65, None, 64)):
        c = Case(900, K, N, R, 5, cols=cols, base=base, f32=f32, seed=R + N)
        runs, index = [1, 300, 63, 64, 128, 2, 200, 65, 77], []
        for n in runs:
            index += [int(torch.randint(-1, 5, (1,), generator=g))] * n
        c.index = torch.tensor(index, dtype=torch.int32)
        out, out32 = c.run(cuda_device)
        c.check(out, out32)
        if base == "bf16":                   # in place: rows without an adapter stay as they are, bit for bit
            y = c.base.to(cuda_device)
            none = (c.index < 0).nonzero()[:, 0].to(cuda_device)
            y.view(torch.int16)[none] = 0x7fab
            c.run(cuda_device)
            dl.linear_adapters(c.x.to(cuda_device), c.adapters(cuda_device), c.index.to(cuda_device), y, out=y,
                               out_f32=torch.empty(900, N, device=cuda_device) if f32 else None)
            some = (c.index >= 0).nonzero()[:, 0].to(cuda_device)
            assert torch.equal(y[some], out[some]) and bool((y.view(torch.int16)[none] == 0x7fab).all())


def test_long_runs_repeat(cuda_device):
    """Bitwise repeatable among other calls, on one workspace of the largest of several token counts."""
    cases = [Case(T, 512, 192, 32, 4, cols=[128, 64], order="runs", none=0.0, seed=T) for T in (300, 5000, 1100)]
    ws = dl.Workspace(dl.adapters_workspace_bytes(5000, cases[0].adapters(cuda_device)))
    args = [(c.x.to(cuda_device), c.adapters(cuda_device), c.index.to(cuda_device), c.base.to(cuda_device)) for c in cases]
    want = [dl.linear_adapters(*a).clone() for a in args]
    for c, w in zip(cases[:1] + cases[2:], want[:1] + want[2:]):
        c.check(w)
    for _ in range(3):
        got = [dl.linear_adapters(*a, workspace=ws) for a in args]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert dl.device_status() == 0


@pytest.mark.parametrize("R", [8, 40, 64, 128, 136])
@pytest.mark.parametrize("base,f32", [("bf16", False), ("fp32", True), (None, False), ("bf16", True)])
def test_mixed_tokens_of_few_adapters(cuda_device, R, base, f32):
    """Many tokens of each adapter, in no order: tiles by lists of tokens, beside long runs and adapters with few."""
    for T, K, N, cols, num in ((700, 520, 192, [128, 64], 3), (1500, 64, 100, None, 9), (400, 1032, 65, None, 1),
                               (1500, 136, 72, None, 1)):
        c = Case(T, K, N, R, num, cols=cols, base=base, f32=f32, seed=R + T)
        g = torch.Generator().manual_seed(R)
        c.index[:] = torch.randint(-1, num, (T,), generator=g).int()
        c.index[100:300] = 0                 # a run, with others of the same adapter left over
        if num > 2:
            c.index[c.index == 2] = 1        # (fewer than enough of one adapter)
            c.index[[5, 50, 350]] = 2
        out, out32 = c.run(cuda_device)
        c.check(out, out32)
        perm = torch.randperm(T, generator=g)       # another order, without the run: to the tolerance alike
        c.x, c.index = c.x[perm], c.index[perm]
        c.base = None if c.base is None else c.base[perm]
        c.check(*c.run(cuda_device))


def test_most_tiles(cuda_device):
    """As many adapters as have just enough tokens for tiles by lists."""
    c = Case(4080, 64, 64, 64, 102, none=0.0, ranks=False)
    c.index = (torch.arange(4080) % 102).int()
    ws = dl.Workspace(dl.adapters_workspace_bytes(4080, c.adapters(cuda_device)))
    c.check(*c.run(cuda_device, workspace=ws))
