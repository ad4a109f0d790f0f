"""block_norm of many long rows through shared memory, in every form that goes there, against its formulas in 64 bits."""
import itertools

import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from step_util import BF16, F32, assert_near, block_norm64
from test_block_norm_gpu import call, check, make, norm_on

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,h", [(1024, "fp32"), (4096, "fp32"), (5120, "bf16"), (8192, "bf16"), (8192, "fp32")])
@pytest.mark.parametrize("post,pre", list(itertools.product([None, "rms", "layer"], ["rms", "layer"])))
@pytest.mark.parametrize("gate", [None, "row", "channel"])
def test_forms(cuda_device, dim, h, post, pre, gate):
    c = make(610, dim, y="fp32" if pre == "rms" else "bf16", h=h, post=post, pre=pre, gate=gate, act="sigmoid" if post else None,
             bias=post == "layer", offset=float(gate == "row"), w="fp32" if gate == "channel" else "bf16", scale=0.25, h_scale=1.5,
             seed=dim)
    check(c, call(c, cuda_device))


@pytest.mark.parametrize("rows", [608, 609, 911, 1217, 3000])
def test_row_counts(cuda_device, rows):
    """One row to a CTA, fewer than stages, more; the same bit for bit in place."""
    c = make(rows, 5120, post="rms", gate="row", h="fp32", h_scale=-0.5, seed=rows)
    want = [t.clone() for t in call(c, cuda_device)]
    check(c, want)
    y, h = c["y"].to(cuda_device), c["h"].to(cuda_device)
    r, x = dl.block_norm(y, h, post=norm_on(c["post"], cuda_device), pre=norm_on(c["pre"], cuda_device),
                         gate=c["gate"].to(cuda_device), h_scale=-0.5, out_h=h, out_x=y)
    assert r is h and x is y and torch.equal(r, want[0]) and torch.equal(x, want[1])


@pytest.mark.parametrize("dim", [2048, 8192])
def test_wide_outputs_and_views(cuda_device, dim):
    """x as wide as y; rows of wider tensors, aligned: what lies between them stays."""
    c = make(700, dim, y="fp32", h="fp32", post="layer", pre="layer", gate="row", act="sigmoid", bias=True, h_scale=2.0)
    wide = lambda t: torch.nn.functional.pad(t.to(cuda_device), (8, 16))[:, 8:8 + dim]   # noqa: E731
    r, x = (torch.full((700, dim + 24), 7.0, dtype=F32, device=cuda_device) for _ in range(2))
    got = dl.block_norm(wide(c["y"]), wide(c["h"]), post=norm_on(c["post"], cuda_device), pre=norm_on(c["pre"], cuda_device),
                        gate=c["gate"].to(cuda_device), gate_act="sigmoid", h_scale=2.0, out_h=r[:, 8:8 + dim], out_x=x[:, 8:8 + dim])
    check(c, got)
    for t in (r, x):
        assert bool((t[:, :8] == 7).all()) and bool((t[:, 8 + dim:] == 7).all())


def off_mean(dim):
    """What a centred value of a row is off by through its mean, beside norm64's 2^-22 max |v|, which no number below fp32's
    normal ones is part of: a mean is a sum of up to dim products v / dim in dim - 1 fused steps and additions, and
    each of these that gives less than 2^-126 is rounded to a multiple of 2^-149, by 2^-150 at most.  The second
    pass takes the first mean's error off and has its own, as large.  (Sums and differences of the values
    themselves are multiples of 2^-149: exact.)"""
    return dim * 2.0 ** -150


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("spread", [1e30, 3e37, 1e-25, 1e-38])
@pytest.mark.parametrize("dim", [2048, 8192])
def test_range(cuda_device, kind, spread, dim):
    """Squares beyond fp32's range, either way, in some rows, in the norm of y and in the stream's."""
    eps = 0.0 if spread < 1 else 1e-6
    for name in ("y", "h"):
        c = make(620, dim, y="fp32", h="fp32", post=kind, pre=kind, eps=eps, seed=dim, scale=0.0 if name == "h" else 1.0)
        c[name][::3] *= spread
        (r, x), (dr, dx) = block_norm64(c["y"], c["h"], c["post"], c["pre"], None, None, c["scale"], 1.0)
        if kind == "layer":
            def part(v, w, dv):          # a norm's error by an error dv of each value, as in block_norm64
                n = v - v.mean(-1, keepdim=True)
                inv = 1 / torch.sqrt(n.square().mean(-1, keepdim=True) + eps)
                return 2 * w.double().abs() * (inv * dv + n.abs() * inv ** 3 * (n.abs() * dv).mean(-1, keepdim=True))

            tiny = torch.full(r.shape, off_mean(dim), dtype=torch.float64)
            more = c["scale"] * part(c["y"].double(), c["post"][1], tiny)
            dr, dx = dr + more, dx + part(r, c["pre"][1], more + tiny)
        got = call(c, cuda_device)
        assert_near(got[0], r, dr, "r")
        assert_near(got[1], x, dx, "x")


def test_rows_keep_to_themselves(cuda_device):
    for dim in (2048, 8192):
        c = make(700, dim, y="bf16", h="fp32", post="rms", gate="row")
        clean = call(c, cuda_device)
        c["y"][3, dim // 2], c["h"][308, 0], c["gate"][612, 0] = float("nan"), float("inf"), float("nan")
        bad = call(c, cuda_device)
        keep = [i for i in range(700) if i not in (3, 308, 612)]
        for a, b in zip(clean, bad):
            assert torch.equal(a[keep], b[keep])
        r, x = (t.cpu().float() for t in bad)
        for i in (3, 612):
            assert bool(torch.isnan(r[i]).all()) and bool(torch.isnan(x[i]).all())
        assert torch.isinf(r[308, 0]) and bool((x[308, 1:] == 0).all()) and torch.isnan(x[308, 0])


def test_outputs_that_are_given(cuda_device):
    """Outputs of either type are the tensors that come back."""
    for rows, dim, h in ((6, 264, "bf16"), (6, 2050, "fp32"), (700, 2048, "fp32")):
        c = make(rows, dim, h=h, post="rms")
        for kind in (BF16, F32):
            r, x = (torch.empty(rows, dim, dtype=kind, device=cuda_device) for _ in range(2))
            got = call(c, cuda_device, out_h=r, out_x=x)
            assert got[0] is r and got[1] is x
            check(c, got)
