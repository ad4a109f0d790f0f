"""linear_adapters with first products next to fp32's largest number, and infinite ones."""
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from step_util import BF16, HALF

pytestmark = pytest.mark.gpu

LARGEST = (2 ** 24 - 1) * 2.0 ** 104     # fp32's; bf16's is 255 * 2^120
# multiples of 2^104, made of terms of at most 8 bits each, so that every sum of some of them is exact: just at and past
# what bf16 rounds to infinity (255.5 * 2^120), in between, next to the largest, the largest
FIRST = [(255, 128, 0), (255, 128, 1), (255, 129, 255), (255, 200, 77), (255, 255, 127), (255, 255, 128), (255, 255, 129),
         (255, 255, 255)]


def make(dev, T, R, b, values, mixed):
    """Token t has adapter t % len(values), whose first product of rank 3 is values[..]; the other ones are zero."""
    num, K = len(values), 64
    A, B = torch.zeros(num, R, K), torch.zeros(num, len(b), R)
    for i, v in enumerate(values):
        for k, n in enumerate(v):
            A[i, 3, 7 * k] = n * 2.0 ** (120 - 8 * k)
    B[:, :, 3] = torch.tensor(b)
    index = torch.arange(T) % num if mixed else torch.arange(T) * num // T
    return (torch.ones(T, K, dtype=BF16, device=dev), dl.Adapters(A.to(BF16).to(dev), B.to(BF16).to(dev)),
            index.int().to(dev), index)


@pytest.mark.parametrize("R", [8, 48])
@pytest.mark.parametrize("T,mixed", [(1, True), (16, True), (100, True), (300, True), (1024, False), (1024, True)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_first_products_beyond_bf16(cuda_device, T, mixed, R, sign):
    """They are finite in fp32, and so is what small weights, or a base of the other sign, make of them.

    Two parts hold 2^-17 of the value, 2^-16 next to the largest; three hold it whole, and products with powers of
    two are exact."""
    b = [2.0 ** -100, -2.0 ** -3, 0.5, 0.0, 1.0, 2.0 ** -126]
    x, ad, on_dev, index = make(cuda_device, T, R, b, [tuple(sign * n for n in v) for v in FIRST], mixed)
    first = torch.tensor([sum(n * 2.0 ** (120 - 8 * k) for k, n in enumerate(v)) for v in FIRST], dtype=torch.float64) * sign
    base = torch.zeros(T, len(b), device=cuda_device)
    base[:, 4] = -sign * 3e38
    want = first[index][:, None] * torch.tensor(b, dtype=torch.float64) + base.cpu().double()
    size = first.abs()[index][:, None] * torch.tensor(b, dtype=torch.float64).abs()
    out32 = torch.empty_like(base)
    for f32 in (False, True):
        out = dl.linear_adapters(x, ad, on_dev, base, out_f32=out32 if f32 else None).cpu().double()
        err = (out - want).abs()
        limit = (2.0 ** -23 if f32 else 2.0 ** -16) * size + HALF[BF16] * want.abs() + 2.0 ** -134
        assert bool(torch.isfinite(out).all()) and bool((err <= limit * (1 + 2.0 ** -8)).all())
    err = (out32.cpu().double() - want).abs()
    assert bool((err <= 2.0 ** -23 * size + 2.0 ** -149).all())


@pytest.mark.parametrize("T,mixed", [(1, True), (16, True), (100, True), (300, True), (1024, False), (1024, True)])
@pytest.mark.parametrize("f32", [False, True])
def test_infinite_first_products(cuda_device, T, mixed, f32):
    """An infinity times a weight that is not zero is one; times zero it is NaN."""
    inf = float("inf")
    b = [2.0 ** -100, -0.5, 2.0, 0.0]
    x, ad, on_dev, index = make(cuda_device, T, 16, b, [(inf,), (-inf,), (1.0,)], mixed)
    out32 = torch.empty(T, 4, device=cuda_device) if f32 else None
    out = dl.linear_adapters(x, ad, on_dev, out_f32=out32)
    first = torch.tensor([inf, -inf, 2.0 ** 120], dtype=torch.float64)[index]
    want = first[:, None] * torch.tensor(b, dtype=torch.float64)
    for got in (out, out32) if f32 else (out,):
        assert torch.equal(got.cpu().double().nan_to_num(7.0), want.nan_to_num(7.0))
