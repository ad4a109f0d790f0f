"""kv_append against a loop in fp32 with separate roundings (bit for bit) and against the
rotation in 64 bits."""
import numpy as np
import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from kv_util import F8, Step, reference_append, rope_tables, same_codes

pytestmark = pytest.mark.gpu


def run(step, dev, rot=None, positions=None, in_place=False, fused=False):
    c = step.cache(dev)
    cos = sin = None
    if rot:
        cos, sin = (torch.tensor(x, device=dev) for x in rope_tables(max(step.lens + [1]) + 5, rot))
    q, k, v = step.q.to(dev), step.new_k.to(dev), step.new_v.to(dev)
    if fused:            # views of one row, as the QKV projection writes it
        row = torch.cat([x.reshape(step.T, -1) for x in (q, k, v)], 1)
        a, b = step.heads * step.dim, step.kv_heads * step.dim
        q, k, v = (x.view(step.T, -1, step.dim) for x in (row[:, :a], row[:, a:a + b], row[:, a + b:]))
    pos = None if positions is None else torch.tensor(positions, dtype=torch.int32, device=dev)
    out = dl.kv_append(q, k, v, c, *step.seqs(dev), max_q=step.max_q, cos=cos, sin=sin, positions=pos,
                       out_q=q if in_place else None)
    torch.cuda.synchronize(dev)
    want = reference_append(step, *(rope_tables(max(step.lens + [1]) + 5, rot) if rot else (None, None)),
                            positions=positions)
    return out, c, want


def check(step, out, c, want):
    q, k, v, ks, vs = want
    assert torch.equal(out.cpu(), torch.tensor(q).bfloat16())
    assert np.array_equal(c.k_scale.cpu().numpy(), ks, equal_nan=True)
    assert np.array_equal(c.v_scale.cpu().numpy(), vs, equal_nan=True)
    assert same_codes(c.k.view(torch.uint8).cpu().numpy(), k)
    assert same_codes(c.v.view(torch.uint8).cpu().numpy(), v)


@pytest.mark.parametrize("heads,kv_heads,dim,rot", [(8, 2, 128, 128), (3, 3, 64, 64), (16, 1, 128, 64),
                                                    (5, 1, 64, 16), (4, 4, 128, None)])
@pytest.mark.parametrize("page,block", [(16, 16), (8, 1), (64, 4), (32, 32), (128, 128), (1024, 256)])
def test_append_matches_the_definition(cuda_device, heads, kv_heads, dim, rot, page, block):
    # inside a begun block, at a block's first slot, over several pages, from nothing, one token
    step = Step([5, 16, 77, 33, 129, 1], [2, 3, 50, 33, 1, 1], heads=heads, kv_heads=kv_heads, dim=dim,
                page=page, block=block, seed=page + block + dim)
    check(step, *run(step, cuda_device, rot))


def test_views_of_one_row_and_in_place_queries(cuda_device):
    step = Step([40, 7], [9, 7], seed=3)
    check(step, *run(step, cuda_device, 128, fused=True))
    check(step, *run(step, cuda_device, 128, in_place=True))
    one = Step([23], [1], seed=4)
    check(one, *run(one, cuda_device, 128, fused=True))


def test_positions_of_the_caller(cuda_device):
    step = Step([40, 30], [4, 6], seed=5)
    check(step, *run(step, cuda_device, 128, positions=[0, 3, 3, 44, 1, 9, 2, 7, 1000, -4]))


def test_block_scale_grows_and_old_codes_follow(cuda_device):
    step = Step([12, 12, 12], [3, 3, 3], seed=6)
    step.new_k *= 64
    step.new_v[3:6] *= 1e-3                      # smaller than the block's scale: it stays
    out, c, want = run(step, cuda_device, 128)
    check(step, out, c, want)
    assert (want[3] != step.k_scale.numpy()).any()


def test_a_new_block_forgets_what_its_slots_held(cuda_device):
    step = Step([16], [16], seed=7)
    step.k = torch.full_like(step.k.view(torch.uint8), 127).view(F8)
    step.k_scale.fill_(float("nan"))
    out, c, want = run(step, cuda_device, 128)
    check(step, out, c, want)
    pg = int(step.table[0, 0])
    assert torch.isfinite(c.k_scale[pg]).all() and torch.isfinite(c.k[pg].float()).all()


def test_extreme_values(cuda_device):
    step = Step([16, 20, 3], [4, 20, 3], seed=8)
    step.new_k[0] = 0
    step.new_v[:4] = 0                           # an all-zero block beside codes: scale stays
    step.new_v[4:] = 0                           # an all-zero new block: the smallest scale
    step.new_k[5, 0, 3] = float("inf")
    step.new_k[6, 1, 70] = float("-inf")
    step.new_k[7, 0, 9] = float("nan")
    step.new_v[25, 0, 1] = 3.3e38
    step.new_v[26, 1, 1] = 1e-38
    check(step, *run(step, cuda_device))


def test_scale_boundary_is_448(cuda_device):
    step = Step([2], [2], seed=9)
    for top in (448.0, 450.0, 224.0, 1.75, 1.7578125):
        step.new_v.clamp_(-1, 1)
        step.new_v[0, 0, 0] = top
        check(step, *run(step, cuda_device))


def test_sequences_without_room(cuda_device):
    """Fewer cached than new tokens: the first ones have no place; an absent page takes nothing."""
    step = Step([3, 0, 20], [5, 2, 6], seed=10)
    step.table[2, 1] = step.pages + 7
    check(step, *run(step, cuda_device, 128))
    step.table[2, 1] = -3
    check(step, *run(step, cuda_device, 128))


def test_no_new_tokens_and_empty_batch(cuda_device):
    step = Step([9, 6], [0, 2], seed=11)
    check(step, *run(step, cuda_device, 128))
    c = step.cache(cuda_device)
    before = c.k.view(torch.uint8).clone()
    none = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device=cuda_device)
    dl.kv_append(None, none, none, c, torch.zeros(0, 1, dtype=torch.int32, device=cuda_device),
                 torch.zeros(0, dtype=torch.int32, device=cuda_device),
                 torch.zeros(1, dtype=torch.int32, device=cuda_device), max_q=0)
    assert torch.equal(before, c.k.view(torch.uint8))


def test_strided_cache_and_keys_only(cuda_device):
    """Keys and values as views of one buffer that holds other layers too."""
    step = Step([30, 11], [14, 11], seed=12)
    P, H, pg, D = step.k.shape
    big = torch.zeros(P, 3, 2, H, pg, D, dtype=torch.uint8, device=cuda_device)
    k, v = big[:, 1, 0], big[:, 1, 1]
    k.copy_(step.k.view(torch.uint8))
    v.copy_(step.v.view(torch.uint8))
    sb = torch.zeros(P, 2, H, pg // step.block + 3, device=cuda_device)
    ks, vs = sb[:, 0, :, :1], sb[:, 1, :, :1]
    ks.copy_(step.k_scale)
    vs.copy_(step.v_scale)
    c = dl.PagedKVCache(k, v, ks, vs)
    assert dl.kv_append(None, step.new_k.to(cuda_device), step.new_v.to(cuda_device), c,
                        *step.seqs(cuda_device), max_q=14) is None
    _, wk, wv, wks, wvs = reference_append(step)
    assert same_codes(k.cpu().numpy(), wk) and same_codes(v.cpu().numpy(), wv)
    assert np.array_equal(ks.cpu().numpy(), wks) and np.array_equal(vs.cpu().numpy(), wvs)
    assert not big[:, 0].any() and not big[:, 2].any() and not sb[..., 1:].any()


def test_rotation_against_64_bits(cuda_device):
    """|x'| error: two products and a sum in fp32 (3 x 2^-24 of |x| + |y|), then bf16 (2^-8)."""
    step = Step([700], [700], heads=2, kv_heads=1, page=64, seed=13)
    out, _, _ = run(step, cuda_device, 128)
    a = np.outer(np.arange(700), 10000.0 ** (-np.arange(0, 128, 2) / 128))
    c, s = np.float32(np.cos(a)).astype(np.float64)[:, None], np.float32(np.sin(a)).astype(np.float64)[:, None]
    x = step.q.double().numpy()
    want = np.concatenate([x[..., :64] * c - x[..., 64:] * s, x[..., 64:] * c + x[..., :64] * s], -1)
    size = np.abs(x[..., :64]) + np.abs(x[..., 64:])
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * np.concatenate([size, size], -1)).all()


def test_another_stream(cuda_device):
    step = Step([64, 50], [20, 31], seed=14)
    side = torch.cuda.Stream(cuda_device)
    side.wait_stream(torch.cuda.current_stream(cuda_device))
    with torch.cuda.stream(side):
        check(step, *run(step, cuda_device, 128))


def test_refusals(cuda_device):
    step = Step([9], [2], seed=15)
    c, seqs = step.cache(cuda_device), step.seqs(cuda_device)
    q, k, v = (x.to(cuda_device) for x in (step.q, step.new_k, step.new_v))
    cos, sin = (torch.tensor(x, device=cuda_device) for x in rope_tables(16, 128))
    ok = dict(max_q=2, cos=cos, sin=sin)
    with pytest.raises(ValueError, match="bfloat16"):
        dl.kv_append(q.float(), k, v, c, *seqs, **ok)
    with pytest.raises(ValueError, match="k must be"):
        dl.kv_append(q, q, v, c, *seqs, **ok)
    with pytest.raises(ValueError, match="same tokens"):
        dl.kv_append(q, k, v[:1], c, *seqs, **ok)
    with pytest.raises(ValueError, match="CUDA"):
        dl.kv_append(q.cpu(), k, v, c, *seqs, **ok)
    with pytest.raises(ValueError, match="int32"):
        dl.kv_append(q, k, v, c, seqs[0], seqs[1].long(), seqs[2], **ok)
    with pytest.raises(ValueError, match="q_start"):
        dl.kv_append(q, k, v, c, seqs[0], seqs[1], seqs[2][:1], **ok)
    with pytest.raises(dl.DLError, match="rotary_dim"):
        dl.kv_append(q, k, v, c, *seqs, max_q=2, cos=cos[:, :4].contiguous(), sin=sin[:, :4].contiguous())
    with pytest.raises(dl.DLError, match="max_q"):
        dl.kv_append(q, k, v, c, *seqs, max_q=-1, cos=cos, sin=sin)
    with pytest.raises(ValueError, match="cos"):
        dl.kv_append(q, k, v, c, *seqs, max_q=2, cos=cos, sin=sin[:3])
    with pytest.raises(dl.DLError, match="multiples of 8"):
        odd = torch.zeros(2, 260, dtype=torch.bfloat16, device=cuda_device)
        dl.kv_append(None, odd[:, :256].view(2, 2, 128), v, c, *seqs, max_q=2)
    bad = dl.PagedKVCache.empty(2, 2, 32, device=cuda_device)
    with pytest.raises(dl.DLError, match="head_dim"):
        dl.kv_append(None, torch.zeros(2, 2, 32, dtype=torch.bfloat16, device=cuda_device),
                     torch.zeros(2, 2, 32, dtype=torch.bfloat16, device=cuda_device), bad, *seqs, max_q=2)
