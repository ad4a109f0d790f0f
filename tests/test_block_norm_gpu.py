"""block_norm against its formulas in 64 bits, element by element."""
import itertools

import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from step_util import BF16, F32, assert_near, block_norm64

pytestmark = pytest.mark.gpu


def make(rows, dim, *, y="bf16", h="fp32", post=None, pre="rms", gate=None, act=None, w="bf16", bias=False, offset=0.0,
         eps=1e-6, scale=1.0, h_scale=1.0, seed=0, spread=1.0, mean=0.0):
    """CPU inputs of a call."""
    g = torch.Generator().manual_seed(seed)
    kinds = {"bf16": BF16, "fp32": F32}
    randn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    c = {"y": None if y is None else (spread * randn(rows, dim) + mean).to(kinds[y]),
         "h": None if h is None else (2 * spread * randn(rows, dim) - mean).to(kinds[h]),
         "act": act, "scale": scale, "h_scale": h_scale, "gate": None}
    if gate is not None:
        shape = {"channel": (dim,), "row": (rows, 1), "full": (rows, dim)}[gate]
        c["gate"] = randn(*shape).to(kinds[w])
    for n, kind in (("post", post), ("pre", pre)):
        c[n] = None if kind is None else (kind, None if w is None else (1 + 0.2 * randn(dim) - offset).to(kinds[w]),
                                          (0.3 * randn(dim)).to(kinds[w or "bf16"]) if bias else None, eps, offset)
    return c


def norm_on(n, dev):
    if n is None:
        return None
    kind, w, b, eps, offset = n
    return dl.Norm(None if w is None else w.to(dev), None if b is None else b.to(dev), kind=kind, eps=eps, offset=offset)


def call(c, dev, **kw):
    on = lambda t: None if t is None else t.to(dev)   # noqa: E731
    return dl.block_norm(on(c["y"]), on(c["h"]), post=norm_on(c["post"], dev), pre=norm_on(c["pre"], dev),
                         gate=on(c["gate"]), gate_act=c["act"], scale=c["scale"], h_scale=c["h_scale"], **kw)


def check(c, got):
    (r, x), (dr, dx) = block_norm64(c["y"], c["h"], c["post"], c["pre"], c["gate"], c["act"], c["scale"], c["h_scale"])
    if got[0] is not None:
        assert_near(got[0], r, dr, "r")
    if got[1] is not None:
        assert_near(got[1], x, dx, "x")


DIMS = [1, 2, 7, 8, 31, 63, 64, 65, 128, 129, 200, 256, 512, 1000, 1024, 1025, 1032, 1537, 2048, 4096, 4104, 5120, 8192,
        8200, 10001, 16384, 16392, 20000, 32760, 32767, 32768]


@pytest.mark.parametrize("dim", DIMS)
def test_widths(cuda_device, dim):
    for k, rows in enumerate((1, 3, 37)):
        c = make(rows, dim, post="rms" if k else None, pre="layer" if k == 2 else "rms", bias=k == 2, seed=dim + rows)
        check(c, call(c, cuda_device))


@pytest.mark.parametrize("post,pre,gate,act", list(itertools.product(
    [None, "rms", "layer"], [None, "rms", "layer"], [None, "channel", "row", "full"], [None, "sigmoid"])))
def test_forms(cuda_device, post, pre, gate, act):
    for i, dim in enumerate((96, 1100, 1537)):
        c = make(5, dim, post=post, pre=pre, gate=gate, act=act, bias=i == 1, offset=float(i == 2), scale=0.25, h_scale=1.5,
                 seed=i, w="fp32" if i == 0 else "bf16")
        check(c, call(c, cuda_device))


@pytest.mark.parametrize("y,h,w", list(itertools.product(["bf16", "fp32", None], ["bf16", "fp32", None], ["bf16", "fp32", None])))
def test_types(cuda_device, y, h, w):
    if y is None and h is None:
        return
    for dim in (264, 2050, 4096):
        c = make(6, dim, y=y, h=h, w=w, post=None if y is None else "rms", seed=dim)
        got = call(c, cuda_device)
        assert (got[0] is None) == (y is None)
        if got[0] is not None:
            assert got[0].dtype == (c["h"] if h else c["y"]).dtype
        check(c, got)
        x = torch.empty(6, dim, device=cuda_device)
        check(c, (None, call(c, cuda_device, out_x=x)[1]))
        assert x.dtype == F32


@pytest.mark.parametrize("rows", [1, 2, 303, 304, 305, 1000, 5000])
def test_row_counts(cuda_device, rows):
    for dim in (40, 130, 1152):
        c = make(rows, dim, post="rms", seed=rows)
        check(c, call(c, cuda_device))


@pytest.mark.parametrize("dim", [1032, 1536, 2048, 4096, 4104, 4608, 5120, 8192, 8200, 16384])
@pytest.mark.parametrize("y,h", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
def test_many_long_rows(cuda_device, dim, y, h):
    """Rows that go through shared memory, several a CTA; the same in place, and with x as wide as y."""
    c = make(700, dim, y=y, h=h, post="rms" if dim % 16 else None, pre="layer" if dim == 4096 else "rms", bias=dim == 2048,
             gate="channel" if dim == 8192 else None, scale=0.5)
    want = [t.clone() for t in call(c, cuda_device)]
    check(c, want)
    ty, th = c["y"].to(cuda_device), c["h"].to(cuda_device)
    kw = dict(post=norm_on(c["post"], cuda_device), pre=norm_on(c["pre"], cuda_device), scale=0.5,
              gate=None if c["gate"] is None else c["gate"].to(cuda_device))
    r, x = dl.block_norm(ty, th, out_h=th, out_x=ty, **kw)
    assert r is th and x is ty and torch.equal(r, want[0])
    check(c, (r, x))


def test_no_rows(cuda_device):
    c = make(0, 64)
    r, x = call(c, cuda_device)
    assert r.shape == x.shape == (0, 64)


@pytest.mark.parametrize("dim", [64, 1030, 2048, 8192])
def test_views(cuda_device, dim):
    """Rows of wider tensors, at offsets that break the wide loads' alignment and at some that do not;
    what lies between the rows stays."""
    for off, extra in ((0, 8), (8, 24), (1, 7), (3, 10)):
        c = make(9, dim, post="rms", gate="full", seed=off)
        wide = lambda t: torch.nn.functional.pad(t.to(cuda_device), (off, extra))   # noqa: E731
        inner = lambda t: t[:, off:off + dim]   # noqa: E731
        y, h, g = (inner(wide(c[n])) for n in ("y", "h", "gate"))
        r, x = (torch.full((9, dim + off + extra), 7.0, dtype=d, device=cuda_device) for d in (F32, BF16))
        got = dl.block_norm(y, h, post=norm_on(c["post"], cuda_device), pre=norm_on(c["pre"], cuda_device), gate=g,
                            out_h=inner(r), out_x=inner(x))
        check(c, got)
        for t in (r, x):
            assert bool((t[:, :off] == 7).all()) and bool((t[:, off + dim:] == 7).all())


def test_side_by_side(cuda_device):
    """An output beside its input in one wider row is no overlap; one that meets it is refused."""
    c = make(6, 256)
    both = torch.cat([c["y"], torch.zeros(6, 256, dtype=BF16)], 1).to(cuda_device)
    got = dl.block_norm(both[:, :256], c["h"].to(cuda_device), pre=norm_on(c["pre"], cuda_device), out_x=both[:, 256:])
    check(c, got)
    with pytest.raises(dl.DLError, match="overlap"):
        dl.block_norm(both[:, :256], c["h"].to(cuda_device), pre=norm_on(c["pre"], cuda_device), out_x=both[:, 128:384])


@pytest.mark.parametrize("dim", [72, 1537, 8192])
def test_in_place(cuda_device, dim):
    c = make(7, dim, h="bf16", post="layer", pre="rms")
    want = [t.clone() for t in call(c, cuda_device)]
    y, h = c["y"].to(cuda_device), c["h"].to(cuda_device)
    r, x = dl.block_norm(y, h, post=norm_on(c["post"], cuda_device), pre=norm_on(c["pre"], cuda_device), out_h=h, out_x=y)
    assert r is h and x is y and torch.equal(h, want[0]) and torch.equal(y, want[1])
    y, h = c["y"].to(cuda_device), c["h"].to(cuda_device)
    dl.block_norm(y, h, post=norm_on(c["post"], cuda_device), pre=norm_on(c["pre"], cuda_device), out_h=y, out_x=h)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("spread", [1e30, 3e37, 1e-25, 1e-38])
def test_range(cuda_device, kind, spread):
    """Squares beyond fp32's range, either way, in some rows of a warp's several and not in others."""
    for dim in (24, 100, 2048):
        c = make(12, dim, y=None, h="fp32", pre=kind, eps=0.0 if spread < 1 else 1e-6, seed=dim)
        c["h"][::3] *= spread
        check(c, call(c, cuda_device))


@pytest.mark.parametrize("rows,dim", [(3, 264), (3, 1537), (3, 2048), (700, 2048)])
def test_far_gates(cuda_device, rows, dim):
    """Sigmoids next to 0, down to fp32's smallest numbers, times values that bring them back; and next to 1.

    The exponential is off by 2 units of 2^-23 or, below 2^-126, of 2^-149; a sum, a quotient and two products
    add 4 roundings: 2^-20 of the gate and 2^-147."""
    gate = torch.tensor([-86.0, -87.5, -88.5, -90.0, -100.0, -103.0, -110.0, -1e30, float("-inf"), 20.0, 90.0, 3e38, float("inf")])
    gate = gate.repeat(dim // 13 + 1)[:dim]
    y = torch.full((rows, dim), 1e30)
    h = torch.zeros(rows, dim)
    r, _ = dl.block_norm(y.to(cuda_device), h.to(cuda_device), gate=gate.to(cuda_device), gate_act="sigmoid", pre=dl.Norm())
    want = torch.sigmoid(gate.double())
    bound = 1e30 * (2.0 ** -20 * want + 2.0 ** -147)
    assert_near(r, (1e30 * want).expand(rows, dim), bound.expand(rows, dim))


def test_far_mean(cuda_device):
    """A mean of 1000 spreads: its rounding errors do not reach the result beyond the inputs' own."""
    for dim in (200, 4096, 30001):
        c = make(4, dim, y=None, pre="layer", spread=0.01, mean=20.0)
        check(c, call(c, cuda_device))


def test_rows_keep_to_themselves(cuda_device):
    """Infinities and NaN of a row reach no other one, and give there what the formulas give."""
    for dim in (16, 300, 2056):
        c = make(20, dim, post="rms", pre="rms", gate="full")
        clean = call(c, cuda_device)
        c["y"][3, dim // 2], c["h"][8, 0], c["gate"][12, dim - 1] = float("nan"), float("inf"), float("inf")
        bad = call(c, cuda_device)
        keep = [i for i in range(20) if i not in (3, 8, 12)]
        for a, b in zip(clean, bad):
            assert torch.equal(a[keep], b[keep])
        r, x = (t.cpu().float() for t in bad)
        assert bool(torch.isnan(r[3]).all()) and bool(torch.isnan(x[3]).all())
        assert torch.isinf(r[8, 0]) and bool((x[8, 1:] == 0).all()) and torch.isnan(x[8, 0])
        assert torch.isinf(r[12, -1]) and bool((x[12, :-1] == 0).all()) and torch.isnan(x[12, -1])


def test_zero_rows(cuda_device):
    c = make(3, 128, y=None, bias=True)
    c["h"][:] = 0
    check(c, call(c, cuda_device))


def test_repeats_and_graphs(cuda_device):
    """Bitwise repeatable; captured and replayed with other values; on another stream and beside others."""
    c = make(33, 4096, post="rms")
    y, h = c["y"].to(cuda_device), c["h"].to(cuda_device)
    post, pre = norm_on(c["post"], cuda_device), norm_on(c["pre"], cuda_device)
    want = dl.block_norm(y, h, post=post, pre=pre)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = dl.block_norm(y, h, post=post, pre=pre, stream=s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, x = dl.block_norm(y, h, post=post, pre=pre)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, want[0]) and torch.equal(x, want[1])
    y.neg_()
    graph.replay()
    again = dl.block_norm(y, h, post=post, pre=pre)
    assert torch.equal(r, again[0]) and torch.equal(x, again[1])


def test_refusals(cuda_device):
    c = make(4, 64)
    y, h = c["y"].to(cuda_device), c["h"].to(cuda_device)
    pre = norm_on(c["pre"], cuda_device)
    for kw, match in ((dict(pre=dl.Norm(torch.ones(65, device=cuda_device))), "pre"), (dict(gate=y[:2]), "gate"),
                      (dict(gate=torch.ones(4, 1)), "gate"), (dict(gate=torch.ones(63, device=cuda_device)), "gate"),
                      (dict(gate_act="tanh"), "gate_act"), (dict(out_h=h[:3]), "out_h"), (dict(out_x=y.half()), "out_x"),
                      (dict(out_x=y.t()), "out_x"), (dict(scale="a"), "scale")):
        with pytest.raises((ValueError, TypeError), match=match):
            dl.block_norm(y, h, **{**dict(pre=pre), **kw})
    with pytest.raises(ValueError, match="h must"):
        dl.block_norm(y, h[:2], pre=pre)
    with pytest.raises(ValueError, match="y must"):
        dl.block_norm(y.half(), h, pre=pre)
    with pytest.raises(ValueError, match="dense"):
        dl.block_norm(torch.empty(64, 4, dtype=BF16, device=cuda_device).t(), h, pre=pre)
    with pytest.raises(dl.DLError):
        dl.block_norm(y, h, pre=pre, gate=y[:1].expand(4, 64))       # rows that share their memory
    with pytest.raises(dl.DLError, match="needs y"):
        dl.block_norm(None, h, post=pre)


@pytest.mark.parametrize("dim", [65, 72, 200, 517, 1001, 8195])
@pytest.mark.parametrize("x32", [False, True])
def test_views_at_any_offset(cuda_device, dim, x32):
    """Rows of bf16 that begin anywhere in wider ones, weights and gates too: what lies around them stays."""
    g = torch.Generator().manual_seed(dim)
    for offset, extra in ((0, 1), (1, 3), (3, 8), (5, 2), (7, 9)):
        c = make(5, dim, h="bf16", post="rms", pre="layer", gate="full", act="sigmoid", bias=True, seed=dim + offset)

        def place(t, dtype=None, fill=float("nan")):
            wide = torch.full((t.shape[0], t.shape[1] + offset + extra), fill, dtype=dtype or t.dtype, device=cuda_device)
            wide[:, offset:offset + t.shape[1]] = t.to(wide)
            return wide, wide[:, offset:offset + t.shape[1]]

        def vector(t):
            wide = torch.full((t.numel() + offset,), float("nan"), dtype=t.dtype, device=cuda_device)
            wide[offset:] = t.to(cuda_device)
            return wide[offset:]

        norms = {n: dl.Norm(vector(c[n][1]), vector(c[n][2]), kind=c[n][0], eps=c[n][3], offset=c[n][4]) for n in ("post", "pre")}
        zero = torch.zeros(5, dim)
        r_wide, r = place(zero, torch.bfloat16, 7.0)
        x_wide, x = place(zero, F32 if x32 else torch.bfloat16, 7.0)
        dl.block_norm(place(c["y"])[1], place(c["h"])[1], **norms, gate=place(c["gate"])[1], gate_act="sigmoid", scale=c["scale"],
                      h_scale=c["h_scale"], out_h=r, out_x=x)
        check(c, (r, x))
        for wide in (r_wide, x_wide):
            assert bool((wide[:, :offset] == 7).all()) and bool((wide[:, offset + dim:] == 7).all())
