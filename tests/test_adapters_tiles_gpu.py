"""linear_adapters with more tiles of 128 tokens than CTAs that take them, more rows of the first factor than one CTA
has columns for, and more tokens than the lists have shared memory for: every token, in 64 bits.
"""
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from step_util import BF16, F32, F64, HALF

pytestmark = pytest.mark.gpu


class Many:
    """Inputs on the device: `num` adapters of `parts` projections of 32 columns each."""

    def __init__(self, dev, T, K, R, num, parts, index, *, base=BF16, ragged=True, seed=0):
        g = torch.Generator(device=dev).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, device=dev, generator=g)   # noqa: E731
        self.R, self.cols, N = R, [32] * parts, 32 * parts
        self.x, self.index = randn(T, K).to(BF16), index.int().to(dev)
        self.a = (randn(num, parts * R, K) * K ** -0.5).to(BF16)
        self.b = (randn(num, N, R) * R ** -0.5).to(BF16)
        self.base = None if base is None else randn(T, N).to(base)
        self.scale = torch.rand(num, device=dev, generator=g) + 0.5
        self.ranks = None
        if ragged:                       # what lies past an adapter's rank reaches nothing
            self.ranks = torch.randint(0, R + 1, (num,), device=dev, generator=g).int()
            past = torch.arange(R, device=dev) >= self.ranks[:, None]
            self.a.view(num, parts, R, K).masked_fill_(past[:, None, :, None], float("nan"))
            self.b.masked_fill_(past[:, None, :], float("nan"))
        self.adapters = dl.Adapters(self.a, self.b, scale=self.scale, ranks=self.ranks, parts=self.cols)

    def run(self, **kw):
        return dl.linear_adapters(self.x, self.adapters, self.index, self.base, **kw)

    def want(self, whole):
        """(out, bound of its error before rounding) in 64 bits; the bound is adapters64's, for all tokens of
        an adapter at once, with 2^-17 for two parts: a first part leaves at most half its step, 2^-8 of the value,
        exactly a part itself; anything less has steps half as large, and is off by 2^-9 of 2^-8."""
        T, K = self.x.shape
        num, N, R = self.b.shape
        out = torch.zeros(T, N, dtype=F64, device=self.x.device) if self.base is None else self.base.double()
        err = 2.0 ** -24 * out.abs()
        ranks = [R] * num if self.ranks is None else self.ranks.tolist()
        scale = self.scale.tolist()
        for i in self.index.unique().tolist():
            if not 0 <= i < num:
                continue
            at, r, s = (self.index == i).nonzero()[:, 0], ranks[i], scale[i]
            x, n0 = self.x[at].double(), 0
            for p, c in enumerate(self.cols):
                A, B = self.a[i, p * R:p * R + r].double(), self.b[i, n0:n0 + c, :r].double()
                low, spread = s * (x @ A.T), abs(s) * (x.abs() @ A.abs().T)
                dlow = (K / 16 + 32) * 2.0 ** -23 * spread + (2.0 ** -23 + (2.0 ** -26 if whole else 2.0 ** -17)) * low.abs()
                out[at, n0:n0 + c] += low @ B.T
                err[at, n0:n0 + c] += dlow @ B.abs().T + (3 * r / 16 + 8) * 2.0 ** -23 * (low.abs() @ B.abs().T)
                n0 += c
        return out, err + 2.0 ** -24 * out.abs()

    def check(self, got, whole=False):
        want, bound = self.want(whole)
        off = (got.double() - want).abs() > bound * (1 + HALF[got.dtype]) + HALF[got.dtype] * want.abs()
        assert bool(torch.isfinite(got).all()) and not bool(off.any()), f"{int(off.sum())} of {off.numel()} outside the bound, " \
            f"tokens {off.any(1).nonzero()[:8, 0].tolist()}"


def dealt(T, num, seed=0):
    """`num` adapters in turn, in no order."""
    return (torch.arange(T) % num)[torch.randperm(T, generator=torch.Generator().manual_seed(seed))]


def in_runs(T, num, n):
    """Runs of n tokens."""
    return torch.arange(T) // n % num


@pytest.mark.parametrize("K", [512, 576, 1088])
def test_second_tiles_of_clusters(cuda_device, K):
    """200 tiles by lists for 153 clusters of two CTAs, which leave their sums where the next tile's copies go."""
    c = Many(cuda_device, 8190, K, 128, 200, 3, dealt(8190, 200), ragged=K == 576)
    ws = dl.Workspace(dl.adapters_workspace_bytes(8190, c.adapters))
    first = c.run(workspace=ws)
    c.check(first)
    for _ in range(5):
        ws.tensor[dl.WORKSPACE_ZERO_BYTES:].fill_(0xff)
        assert torch.equal(c.run(workspace=ws), first)
    assert dl.device_status() == 0


@pytest.mark.parametrize("K", [64, 192, 448])
def test_second_tiles_of_one_cta(cuda_device, K):
    """400 tiles by lists for 305 CTAs, in fewer steps of 64 k than there are stages, and in more."""
    c = Many(cuda_device, 16400, K, 128, 400, 3, dealt(16400, 400))
    c.check(c.run())
    assert dl.device_status() == 0


@pytest.mark.parametrize("parts,K", [(3, 512), (8, 512), (8, 200)])
def test_runs_then_lists(cuda_device, parts, K):
    """Tiles of tokens in a row, then tiles by lists, of the same CTAs."""
    runs, rest = in_runs(60 * 64, 60, 64), 60 + dealt(100 * 42, 100)
    c = Many(cuda_device, 60 * 64 + 100 * 42, K, 128, 160, parts, torch.cat([rest[:2000], runs, rest[2000:]]))
    c.check(c.run())
    assert dl.device_status() == 0


@pytest.mark.parametrize("parts", [3, 8])
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("base,f32", [(BF16, False), (F32, True), (None, True)])
def test_many_rows_of_the_first_factor(cuda_device, parts, mixed, base, f32):
    """384 and 1024 rows: two and four groups of up to 256 columns, K shared by a cluster."""
    for T, K, R in ((600, 1024, 128), (300, 520, 128), (900, 2048, 104)):
        c = Many(cuda_device, T, K, R, 3, parts, dealt(T, 3) if mixed else in_runs(T, 3, 100), base=base, seed=T)
        out32 = torch.empty(T, 32 * parts, device=cuda_device) if f32 else None
        out = c.run(out_f32=out32)
        c.check(out, f32)
        if f32:
            c.check(out32, True)
            assert torch.equal(out, out32.to(BF16))
    assert dl.device_status() == 0


@pytest.mark.parametrize("T", [8191, 8192, 8193, 20011])
@pytest.mark.parametrize("order", ["mixed", "runs", "singles"])
def test_many_tokens(cuda_device, T, order):
    """The runs' starts in shared memory, and in the workspace; every token a run of its own, tokens without an
    adapter among them; many adapters with few tokens each."""
    num = 3000 if order == "singles" else 60
    index = in_runs(T, num, 97) if order == "runs" else dealt(T, num, T)
    index[5000:5400] = -1
    index[::1009] = -1
    c = Many(cuda_device, T, 128, 16, num, 2, index, seed=T)
    c.check(c.run())
    assert dl.device_status() == 0
