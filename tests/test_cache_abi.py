"""The cached-attention entry points reject bad arguments before any CUDA call (no GPU needed),
and the Python calls refuse what is not a CUDA tensor."""
import ctypes

import pytest
import torch

import weight_streaming_skinny_gb300 as dl

# fake, well-aligned device addresses: never dereferenced, validation fails first
K, V, KS, VS, Q, NK, NV, OUT, COS, SIN, TAB, LEN, ST, WS = (0x100000 * (i + 1) for i in range(14))
vp, ll, i, f, sz = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


def cache(**kw):
    d = dict(k=K, v=V, k_scale=KS, v_scale=VS, page_stride=2 * 64 * 128, head_stride=64 * 128, scale_page_stride=8,
             scale_head_stride=4, num_pages=10, num_heads=2, page_size=64, head_dim=128, block=16)
    d.update(kw)
    return dl._KVCache(*(d[n] for n, _ in dl._KVCache._fields_))


def append(c=None, q=Q, k=NK, v=NV, qs=1024, ks=256, vs=256, out=OUT, cos=COS, sin=SIN, rot=128, pos=99, table=TAB,
           cols=4, lens=LEN, start=ST, batch=2, tokens=5, heads=8, max_q=3):
    fn = dl.load().dl_kv_append
    fn.argtypes = [vp, vp, vp, vp, ll, ll, ll, vp, vp, vp, i, i, vp, vp, i, vp, vp, i, i, i, i, vp]
    c = cache() if c is None else c
    return fn(ctypes.byref(c) if c else None, q, k, v, qs, ks, vs, out, cos, sin, rot, pos, None, table, cols, lens,
              start, batch, tokens, heads, max_q, None)


def attention(c=None, q=Q, qs=1024, out=OUT, lse=None, table=TAB, cols=4, lens=LEN, start=ST, batch=2, tokens=5, heads=8,
              max_q=3, ws=WS):
    fn = dl.load().dl_attention_paged
    fn.argtypes = [vp, vp, ll, vp, vp, vp, i, vp, vp, i, i, i, i, f, vp, sz, vp]
    c = cache() if c is None else c
    return fn(ctypes.byref(c) if c else None, q, qs, out, lse, table, cols, lens, start, batch, tokens, heads, max_q, 0.1,
              ws, 1 << 30, None)


def verify(drafts=Q, probs=K, target=V, kind=0, u=KS, un=VS, tokens=OUT, count=TAB, batch=2, n=3, vocab=100):
    fn = dl.load().dl_verify_draft
    fn.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, vp, i, i, i, vp]
    return fn(drafts, probs, target, kind, u, un, None, tokens, count, batch, n, vocab, None)


CACHE_FAULTS = [(dict(k=None), 1), (dict(v_scale=None), 1), (dict(num_pages=0), 2), (dict(num_heads=0), 2),
                (dict(head_dim=96), 2), (dict(page_size=24), 2), (dict(page_size=4), 2), (dict(page_size=2048), 2),
                (dict(block=3), 2), (dict(block=128), 2), (dict(page_stride=100), 1), (dict(head_stride=64 * 128 + 8), 1),
                (dict(head_stride=1024), 1), (dict(scale_head_stride=1), 1), (dict(k=K + 8), 3), (dict(k_scale=KS + 2), 3)]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_bad_caches(fault, status):
    assert append(cache(**fault)) == status
    assert attention(cache(**fault)) == status
    assert dl.load().dl_last_error() != b""


@pytest.mark.parametrize("fault,status", [
    (dict(c=0), 1), (dict(k=None), 1), (dict(out=None), 1), (dict(q=None), 1), (dict(sin=None), 1), (dict(rot=24), 2),
    (dict(rot=256), 2), (dict(pos=0), 2), (dict(heads=0), 2), (dict(qs=1000), 1), (dict(ks=252), 1), (dict(vs=128), 1),
    (dict(k=NK + 2), 3), (dict(cos=COS + 4), 3), (dict(table=None), 1), (dict(cols=0), 1), (dict(batch=-1), 1),
    (dict(tokens=-5), 1), (dict(max_q=-1), 1), (dict(lens=LEN + 2), 3), (dict(start=None), 1)])
def test_append_arguments(fault, status):
    assert append(**fault) == status


@pytest.mark.parametrize("fault,status", [
    (dict(c=0), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(heads=7), 2), (dict(heads=0), 2), (dict(heads=258), 2),
    (dict(qs=1020), 1), (dict(qs=512), 1), (dict(q=Q + 8), 3), (dict(lse=KS + 2), 3), (dict(ws=None), 4),
    (dict(ws=WS + 16), 3), (dict(table=None), 1), (dict(batch=-2), 1), (dict(max_q=-3), 1), (dict(start=ST + 1), 3)])
def test_attention_arguments(fault, status):
    assert attention(**fault) == status


@pytest.mark.parametrize("fault,status", [
    (dict(kind=2), 1), (dict(batch=-1), 1), (dict(n=64), 2), (dict(n=-1), 2), (dict(vocab=0), 2),
    (dict(vocab=(1 << 18) + 1), 2), (dict(target=None), 1), (dict(drafts=None), 1), (dict(u=None), 1), (dict(un=None), 1),
    (dict(tokens=None), 1), (dict(count=None), 1), (dict(target=V + 2), 3), (dict(kind=1, target=V + 1), 3),
    (dict(tokens=OUT + 2), 3)])
def test_verify_arguments(fault, status):
    assert verify(**fault) == status


def test_nothing_to_do_is_no_call():
    """No sequences, no tokens or no new ones: done without touching the device."""
    assert append(batch=0) == append(tokens=0) == append(max_q=0) == 0
    assert attention(batch=0) == attention(tokens=0) == attention(max_q=0) == 0
    assert verify(batch=0) == 0


def test_workspace_sizes_out_of_range():
    lib = dl.load()
    for bad in ((-1, 1, 8, 2, 128, 1), (1, 1, 7, 2, 128, 1), (1, 1, 8, 2, 100, 1), (1, 1, 0, 1, 128, 1), (1, 1, 8, 2, 128, -1)):
        assert lib.dl_attention_workspace_bytes(*bad) == 0


def test_descriptor_layout():
    assert ctypes.sizeof(dl._KVCache) == 4 * 8 + 4 * 8 + 5 * 4 + 4
    assert dl._KVCache.num_pages.offset == 64


def test_cpu_tensors_are_refused():
    with pytest.raises(ValueError, match="CUDA"):
        dl.PagedKVCache.empty(2, 2, 128, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        dl.verify_draft(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2, 8), torch.zeros(1, 1), torch.zeros(1))
    with pytest.raises(TypeError, match="torch.Tensor"):
        dl.PagedKVCache(1, 2, 3, 4)
