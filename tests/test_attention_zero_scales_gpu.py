"""attention_paged: tokens whose values have a zero scale take weight and nothing else."""
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import Step, reference

pytestmark = pytest.mark.gpu

#: A bf16 rounding alone leaves a relative 2-norm error of about 1.65e-3; probabilities of 11 bits add
#: at most 2^-11 = 4.9e-4 to it, were every error in the same direction.
RMS = 2.5e-3


def run(step, dev):
    lse = torch.empty(step.T, step.heads, device=dev)
    out = dl.attention_paged(step.q.to(dev), step.cache(dev), *step.seqs(dev), max_q=step.max_q, out_lse=lse)
    torch.cuda.synchronize(dev)
    assert dl.device_status() == 0
    return out.double().cpu(), lse.double().cpu()


def check(step, dev):
    want, want_lse, _, _ = reference(step)
    got, lse = run(step, dev)
    assert torch.isfinite(got).all()
    assert (got - want).norm() / want.norm() < RMS
    assert ((lse - want_lse).abs() <= 1e-4 + 1e-5 * want_lse.abs()).all()


@pytest.mark.parametrize("group,news", [(8, 1), (8, 2), (8, 4), (8, 6), (8, 8)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("exponent", [-9, -18, -22, -30, -50])
def test_other_values_keep_their_precision(cuda_device, group, news, dim, exponent):
    """Every second block of values has a zero scale, or one below the smallest that counts; the
    others' scales are small too, down to near that bound."""
    step = Step([300, 77], [news, news], heads=group, kv_heads=1, dim=dim, page=16, block=4, seed=news)
    step.v_scale.fill_(2.0 ** exponent)
    step.v_scale[:, :, ::2] = 0
    step.v_scale[1::2, :, 2] = 2.0 ** -61
    v = step.v_scale.clone()
    step.v_scale[v < 2.0 ** -60] = 0                       # as the reference has it
    want, want_lse, _, _ = reference(step)
    step.v_scale = v
    got, lse = run(step, cuda_device)
    assert torch.isfinite(got).all()
    assert (got - want).norm() / want.norm() < RMS
    assert ((lse - want_lse).abs() <= 1e-4 + 1e-5 * want_lse.abs()).all()


@pytest.mark.parametrize("news", [1, 6])
def test_whole_tiles_of_zero_scales(cuda_device, news):
    """Tiles in which no value counts, before and after those in which some do."""
    step = Step([700, 520], [news, news], heads=8, kv_heads=1, page=64, block=16, seed=3)
    step.v_scale.mul_(2.0 ** -16)
    for b, n in enumerate(step.lens):
        for j in list(range(0, 256, 64)) + list(range(448, n, 64)):
            step.v_scale[int(step.table[b, j // 64])] = 0
    check(step, cuda_device)


def test_nothing_but_zero_scales(cuda_device):
    step = Step([300], [2], seed=4)
    step.v_scale.zero_()
    want_lse = reference(step)[1]
    got, lse = run(step, cuda_device)
    assert not got.any()
    assert ((lse - want_lse).abs() <= 1e-4 + 1e-5 * want_lse.abs()).all()


@pytest.mark.parametrize("group,news", [(8, 1), (8, 2), (8, 4), (8, 6), (8, 8)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("at", ["past", "new"])
def test_a_nan_code_of_zero_scale_is_nan(cuda_device, group, news, dim, at):
    """NaN times zero, as a quantiser leaves it that divides by the largest finite value of a block
    without one: every row that sees the token has a NaN there, and no other."""
    step = Step([140], [news], heads=group, kv_heads=1, dim=dim, page=16, block=1, seed=news)
    j = 131 if at == "past" else 140 - (news + 1) // 2
    p, o = step.slots(0, 140)[j]
    step.v_scale[p, 0, o] = 0
    step.v[p, 0, o] = torch.zeros(dim).to(step.v.dtype)
    want = reference(step)[0]
    step.v.view(torch.uint8)[p, 0, o, 37] = 0xff
    got, _ = run(step, cuda_device)
    first = max(j - (140 - news), 0)                        # the first new token that sees it
    nan = torch.isnan(got)
    assert nan[first:, :, 37].all() and nan.sum() == (news - first) * group
    got[first:, :, 37] = want[first:, :, 37]
    assert (got - want).norm() / want.norm() < RMS
