"""block_norm, linear_adapters and the pages of the cache reject bad arguments before any CUDA call, and
the Python calls refuse what is not a CUDA tensor (no GPU needed)."""
import ctypes

import pytest
import torch

import weight_streaming_skinny_gb300 as dl

# fake, well-aligned device addresses: never dereferenced, validation fails first
Y, H, G, R, X, W, B, IDX, WS, REFS, TAB, LENS, LA, LB, DONE = (0x1000000 * (i + 1) for i in range(15))
vp, ll, i, f, sz = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class Rows(ctypes.Structure):
    _fields_ = [("data", vp), ("stride", ll), ("dtype", i)]


def ref(s):
    return None if s is None else ctypes.byref(s)


def norm(kind=1, w=W, b=None, eps=1e-6, offset=0.0, dtype=0):
    return dl._Norm(w, b, eps, offset, kind, dtype)


def block_norm(y=(Y, 64, 0), h=(H, 64, 0), post=None, pre="rms", gate=None, kind=0, act=0, scale=1.0, h_scale=1.0,
               r=(R, 64, 0), x=(X, 64, 0), rows=4, dim=64):
    fn = dl.load().dl_block_norm
    fn.argtypes = [vp, vp, vp, i, i, f, vp, f, vp, vp, vp, i, i, vp]
    t = [None if v is None else Rows(*v) for v in (y, gate, h, r, x)]
    pre = norm() if pre == "rms" else pre
    return fn(ref(t[0]), ref(post), ref(t[1]), kind, act, scale, ref(t[2]), h_scale, ref(pre), ref(t[3]), ref(t[4]), rows,
              dim, None)


INF = float("inf")


@pytest.mark.parametrize("fault,status", [
    (dict(rows=-1), 1), (dict(dim=0), 2), (dict(dim=32769), 2), (dict(kind=4), 1), (dict(kind=-1), 1), (dict(act=2), 1),
    (dict(y=None, h=None), 1), (dict(kind=1), 1), (dict(y=None, gate=(G, 1, 0), kind=1), 1), (dict(r=None, x=None), 1),
    (dict(x=None), 1), (dict(y=None, post=norm()), 1), (dict(post=norm(kind=3)), 1), (dict(pre=norm(dtype=2)), 1),
    (dict(pre=norm(eps=-1e-6)), 1), (dict(pre=norm(eps=float("nan"))), 1), (dict(pre=norm(offset=INF)), 1),
    (dict(pre=norm(w=W + 1)), 3), (dict(pre=norm(w=W + 2, dtype=1)), 3), (dict(scale=INF), 1), (dict(h_scale=-INF), 1),
    (dict(y=(Y, 63, 0)), 1), (dict(y=(Y, -64, 0)), 1), (dict(y=(Y, 64, 2)), 1), (dict(h=(H + 1, 64, 0)), 3),
    (dict(h=(H + 2, 64, 1)), 3), (dict(gate=(G, 0, 0), kind=3), 1), (dict(gate=(G, 32, 0), kind=3), 1),
    (dict(r=(Y + 2, 64, 0)), 1), (dict(r=(Y, 128, 0)), 1), (dict(r=(H, 64, 1)), 1), (dict(r=(X + 4, 64, 0)), 1),
    (dict(x=(G, 64, 0), gate=(G, 64, 0), kind=3), 1), (dict(x=(W - 4 * 64 * 2 + 2, 64, 0)), 1),
    (dict(x=(R, 64, 0)), 1)])
def test_block_norm_arguments(fault, status):
    assert block_norm(**fault) == status
    assert dl.load().dl_last_error() != b""


def test_no_rows_is_no_call():
    assert block_norm(rows=0) == 0


def adapters(a=W, b=B, scale=None, ranks=None, num=4, rank=16, K=64, N=96, parts=(32, 96)):
    return dl._Adapters(a, b, scale, ranks, num, rank, K, N, len(parts), (ctypes.c_int * 8)(*parts[:8]))


def linear(ad=None, x=(X, 64, 0), index=IDX, base=(G, 96, 0), y=(Y, 96, 0), y32=None, tokens=5, ws=WS, nbytes=1 << 30):
    fn = dl.load().dl_linear_adapters
    fn.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, sz, vp]
    ad = adapters() if ad is None else ad
    t = [None if v is None else Rows(*v) for v in (x, base, y, y32)]
    return fn(ref(ad) if ad else None, ref(t[0]), index, ref(t[1]), ref(t[2]), ref(t[3]), tokens, ws, nbytes, None)


@pytest.mark.parametrize("fault,status", [
    (dict(a=None), 1), (dict(b=None), 1), (dict(a=W + 8), 3), (dict(b=B + 2), 3), (dict(scale=LA + 2), 3), (dict(ranks=LA + 1), 3),
    (dict(num=0), 2), (dict(num=16385), 2), (dict(rank=0), 2), (dict(rank=12), 2), (dict(rank=264), 2), (dict(K=60), 2),
    (dict(K=0), 2), (dict(N=0), 2), (dict(parts=()), 2), (dict(parts=(32, 95)), 2), (dict(parts=(30, 96)), 2),
    (dict(parts=(96, 96)), 2), (dict(parts=(48, 32, 96)), 2), (dict(parts=(112, 96)), 2)])
def test_bad_adapters(fault, status):
    assert linear(adapters(**fault)) == status
    assert dl.load().dl_last_error() != b""


@pytest.mark.parametrize("fault,status", [
    (dict(ad=0), 1), (dict(tokens=-1), 1), (dict(x=None), 1), (dict(index=None), 1), (dict(y=None), 1), (dict(x=(X, 64, 1)), 1),
    (dict(y=(Y, 96, 1)), 1), (dict(y32=(R, 96, 0)), 1), (dict(x=(X, 60, 0)), 1), (dict(x=(X, 68, 0)), 3),
    (dict(x=(X + 8, 64, 0)), 3), (dict(base=(G, 95, 0)), 1), (dict(base=(G, 96, 7)), 1), (dict(y=(Y + 1, 96, 0)), 3),
    (dict(index=IDX + 2), 3), (dict(ws=None), 4), (dict(ws=WS + 16), 3), (dict(nbytes=1000), 4), (dict(y=(G + 2, 96, 0)), 1),
    (dict(y=(G, 192, 0)), 1), (dict(y=(X, 96, 0)), 1), (dict(y32=(Y, 96, 1)), 1), (dict(y32=(G, 96, 1)), 1)])
def test_linear_adapters_arguments(fault, status):
    assert linear(**fault) == status


def test_no_tokens_is_no_call():
    assert linear(tokens=0) == 0


def test_adapters_workspace():
    fn = dl.load().dl_adapters_workspace_bytes
    for bad in ((-1, 4, 16, 1), (1, 0, 16, 1), (1, 20000, 16, 1), (1, 4, 4, 1), (1, 4, 512, 1), (1, 4, 16, 0), (1, 4, 16, 9)):
        assert fn(*bad) == 0
    sizes = [fn(t, 64, 32, 3) for t in (0, 1, 16, 255, 256, 257, 5000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] >= dl.WORKSPACE_ZERO_BYTES
    assert linear(nbytes=fn(5, 4, 16, 2) - 1) == 4


def pool(refs=REFS, table=TAB, lens=LENS, num_pages=10, page_size=64, rows=8, cols=4, caches=1, dev=W, **kw):
    d = dict(k=Y, v=H, k_scale=G, v_scale=R, page_stride=2 * 64 * 128, head_stride=64 * 128, scale_page_stride=8,
             scale_head_stride=4, num_pages=10, num_heads=2, page_size=64, head_dim=128, block=16)
    n = max(caches, 1)
    arr = (dl._KVCache * n)(*[dl._KVCache(*({**d, **(kw if j == n - 1 else {})}[k] for k, _ in dl._KVCache._fields_))
                              for j in range(n)])
    p = dl._KVPages(arr if caches else None, dev, refs, table, lens, max(caches, 0) or caches, num_pages, page_size, rows, cols)
    p.keep = arr
    return p


def call(what, p=None, a=LA, b=LB, done=DONE, n=3, ws=WS, nbytes=1 << 30):
    lib = dl.load()
    for name, types in (("dl_kv_free", [vp, vp, i, vp]), ("dl_kv_compact", [vp, vp, vp, sz, vp]),
                        ("dl_kv_reserve", [vp, vp, vp, vp, i, vp, sz, vp]), ("dl_kv_fork", [vp, vp, vp, vp, i, vp, sz, vp])):
        getattr(lib, name).argtypes = types
    p = pool() if p is None else p
    r = ref(p) if p else None
    if what == "free":
        return lib.dl_kv_free(r, a, n, None)
    if what == "compact":
        return lib.dl_kv_compact(r, done, ws, nbytes, None)
    return getattr(lib, "dl_kv_" + what)(r, a, b, done, n, ws, nbytes, None)


ALL = ["free", "reserve", "fork", "compact"]


@pytest.mark.parametrize("fault,status", [
    (dict(refs=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(refs=REFS + 2), 3), (dict(num_pages=0), 2),
    (dict(page_size=24), 2), (dict(page_size=4), 2), (dict(page_size=2048), 2), (dict(rows=0), 2), (dict(rows=16385), 2),
    (dict(cols=0), 1), (dict(cols=1 << 26), 2), (dict(caches=-1), 1)])
def test_bad_pools(fault, status):
    for what in ALL:
        assert call(what, pool(**fault)) == status
        assert dl.load().dl_last_error() != b""


@pytest.mark.parametrize("fault,status", [
    (dict(caches=2, num_heads=1), 1), (dict(caches=2, head_dim=64), 1), (dict(caches=2, block=8, scale_head_stride=8, scale_page_stride=16), 1),
    (dict(caches=3, k=Y + 8), 3), (dict(caches=1, num_pages=11), 1), (dict(num_pages=11, caches=2), 1),
    (dict(caches=2, v=None), 1), (dict(dev=None), 1), (dict(dev=W + 4), 3)])
def test_bad_caches_of_a_pool(fault, status):
    if fault.get("num_pages") == 11 and fault["caches"] == 1:
        p = pool()
        p.num_pages = 11
    else:
        p = pool(**fault)
    for what in ("fork", "compact"):
        assert call(what, p) == status


@pytest.mark.parametrize("what,fault,status", [
    ("free", dict(p=0), 1), ("free", dict(a=None), 1), ("free", dict(n=-1), 1), ("free", dict(n=9), 1), ("free", dict(a=LA + 1), 3),
    ("reserve", dict(p=0), 1), ("reserve", dict(b=None), 1), ("reserve", dict(done=None), 1), ("reserve", dict(n=9), 1),
    ("reserve", dict(b=LB + 2), 3), ("reserve", dict(ws=None), 4), ("reserve", dict(ws=WS + 16), 3),
    ("reserve", dict(nbytes=100), 4), ("fork", dict(a=None), 1), ("fork", dict(done=DONE + 2), 3), ("fork", dict(nbytes=0), 4),
    ("fork", dict(n=9), 1), ("compact", dict(p=0), 1), ("compact", dict(done=None), 1), ("compact", dict(done=DONE + 1), 3),
    ("compact", dict(ws=None), 4), ("compact", dict(nbytes=1 << 16), 4)])
def test_list_arguments(what, fault, status):
    assert call(what, **fault) == status


def test_empty_lists_are_no_call():
    assert call("free", n=0) == call("reserve", n=0) == call("fork", n=0) == 0


def test_a_table_too_large():
    """What all rows can ask for together is below 2^31."""
    lib = dl.load()
    for rows, cols, status in ((16384, 1 << 17, 2), (16384, (1 << 17) - 1, 4), (9, 1 << 20, 4)):
        for what in ("reserve", "fork"):
            assert call(what, pool(rows=rows, cols=cols), nbytes=0) == status
    assert b"bytes" in lib.dl_last_error()


def test_pages_workspace():
    fn = dl.load().dl_kv_pages_workspace_bytes
    assert fn(0, 1) == fn(1, 0) == fn(1, 16385) == fn((1 << 28) + 1, 1) == 0
    assert fn(10, 8) >= dl.WORKSPACE_ZERO_BYTES


def test_descriptor_layouts():
    assert ctypes.sizeof(dl._Norm) == 32 and dl._Norm.kind.offset == 24
    assert ctypes.sizeof(dl._Adapters) == 4 * 8 + 5 * 4 + 8 * 4 + 4 and dl._Adapters.part_end.offset == 52
    assert ctypes.sizeof(dl._KVPages) == 5 * 8 + 5 * 4 + 4 and dl._KVPages.rows.offset == 52


def test_cpu_tensors_are_refused():
    t = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dl.block_norm(t, t)
    with pytest.raises(TypeError, match="torch.Tensor"):
        dl.block_norm(None, None)
    with pytest.raises(ValueError, match="CUDA"):
        dl.Norm(t[0])
    with pytest.raises(ValueError, match="rms"):
        dl.Norm(kind="batch")
    with pytest.raises(ValueError, match="CUDA"):
        dl.Adapters(t[None], t[None])
    ints = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dl.PagePool([], ints[None], ints[:1], ints, page_size=64)
    with pytest.raises(TypeError, match="PagedKVCache"):
        dl.PagePool([1], ints[None], ints[:1], ints)
