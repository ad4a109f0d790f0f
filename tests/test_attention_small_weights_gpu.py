"""attention_paged: small weights count where the token that has nearly all weight has no value.

A probability goes into the product with the values as an fp16 number (11 significant bits) of a
range in which the row's largest weighted probability is 2^9 at least, and nothing but that
rounding is lost: a weight of 2^-m of the largest is off by at most 2^-11 of itself or, where it is
subnormal, by half of 2^-24, 2^(m - 34) of itself.
"""
import math

import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import F8, Step, reference

pytestmark = pytest.mark.gpu

ROWS = [(8, 1), (8, 2), (8, 4), (8, 6), (8, 8)]      # query heads of one key/value head, new tokens


def limit(m):
    """The relative error of outputs that tokens of weight 2^-m make: the output's rounding to bf16,
    the weights', and 2^-14 for scores and exponentials in fp32 (2^-22 of scores below 2^6, and more)."""
    return 2.0 ** -9 + 2.0 ** -11 + 2.0 ** -14 + 2.0 ** (m - 34)


def sink(group, news, dim, m, classes, tokens=1000, seed=0):
    """One sequence: token 0 has score 0 and zero codes as values; the others have scores of
    -m ln 2 times 1, 62/64 or 60/64 (as many of them as `classes`) and positive values."""
    step = Step([tokens], [news], heads=group, kv_heads=1, dim=dim, page=64, block=16, seed=seed)
    step.q = torch.ones_like(step.q)
    kind = torch.randint(0, classes, (step.pages, 1, step.page, 1), generator=step.g)
    step.k = (-32.0 + 2.0 * kind).expand(step.k.shape).to(F8).contiguous()
    step.v = torch.randint(64, 449, step.v.shape, generator=step.g).float().to(F8)
    p, o = step.slots(0, 1)[0]
    step.k[p, 0, o] = torch.full((dim,), 32.0).to(F8)
    step.v[p, 0, o] = torch.zeros(dim).to(F8)
    step.k_scale.fill_(1)
    step.v_scale.fill_(2.0 ** -6)
    return step, m * math.log(2) / (64 * dim)


def run(step, scale, dev, sequences):
    """The same sequence many times: a CTA then goes through all of its tiles."""
    want = reference(step, scale)[0]
    n = step.T
    table = step.table.expand(sequences, -1).contiguous().to(dev)
    lens = torch.full((sequences,), step.lens[0], dtype=torch.int32, device=dev)
    start = torch.arange(sequences + 1, dtype=torch.int32, device=dev) * n
    q = step.q.to(dev).repeat(sequences, 1, 1)
    out = dl.attention_paged(q, step.cache(dev), table, lens, start, max_q=n, scale=scale)
    torch.cuda.synchronize(dev)
    assert dl.device_status() == 0
    return out.double().cpu().view(sequences, n, step.heads, step.dim), want


@pytest.mark.parametrize("group,news", ROWS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("m", [12, 18, 22, 25, 28])
def test_weights_far_below_the_largest(cuda_device, group, news, dim, m):
    step, scale = sink(group, news, dim, m, 3, seed=m)
    got, want = run(step, scale, cuda_device, 400)
    err = (got - want).flatten(1).norm(dim=1) / want.norm()
    assert err.max() < limit(m), err.max()


@pytest.mark.parametrize("group,news", ROWS)
@pytest.mark.parametrize("dim", [64, 128])
def test_every_part_of_a_weight_counts(cuda_device, group, news, dim):
    """All but one token have the same weight, so nothing averages its rounding out: weights
    over one binade, whose bits beyond the sixth would show if they were left out."""
    for i in range(8):
        m = 10 + (i + 0.5) / 8
        step, scale = sink(group, news, dim, m, 1, tokens=500, seed=i)
        got, want = run(step, scale, cuda_device, 3)
        err = (got - want).flatten(1).norm(dim=1) / want.norm()
        assert err.max() < limit(m), (m, err.max())
