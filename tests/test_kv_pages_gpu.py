"""kv_free, kv_reserve, kv_fork and kv_compact against the same steps on Python lists: the state exactly, and
what every page holds."""
import random

import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from step_util import Pool

pytestmark = pytest.mark.gpu


class Both:
    """A pool on the device, with caches of `layers`, and its Python form; every token's slot of a page
    holds codes of its own in every cache, so that contents say where they came from."""

    def __init__(self, dev, num_pages=40, page=16, rows=8, cols=6, layers=2, heads=2, dim=64, block=4, strided=False):
        self.dev = dev
        self.ref = Pool(num_pages, page, rows, cols)
        self.caches = []
        g = torch.Generator(device=dev).manual_seed(num_pages)
        for _ in range(layers):
            if strided:              # keys and values of a page side by side in one buffer
                kv = torch.randint(0, 256, (num_pages, 2, heads, page, dim), dtype=torch.uint8, device=dev, generator=g)
                s = torch.rand(num_pages, 2, heads, page // block + 1, device=dev, generator=g)[..., :page // block]
                self.caches.append(dl.PagedKVCache(kv[:, 0], kv[:, 1], s[:, 0], s[:, 1]))
            else:
                k, v = (torch.randint(0, 256, (num_pages, heads, page, dim), dtype=torch.uint8, device=dev, generator=g)
                        for _ in range(2))
                ks, vs = (torch.rand(num_pages, heads, page // block, device=dev, generator=g) for _ in range(2))
                self.caches.append(dl.PagedKVCache(k, v, ks, vs))
        if layers:
            self.pool = dl.PagePool.empty(self.caches, rows, cols)
        else:
            z = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)   # noqa: E731
            self.pool = dl.PagePool([], z(rows, cols) - 1, z(rows), z(num_pages), page_size=page)

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.dev)

    def contents(self):
        return [[t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)] for c in self.caches]

    def check(self, before, copies):
        """The state, and every cache after `copies` (from, to, tokens) of what was there before."""
        assert self.pool.refs.tolist() == self.ref.refs
        assert self.pool.seq_lens.tolist() == self.ref.lens
        assert self.pool.block_table.tolist() == self.ref.table
        if {s for s, _, _ in copies} & {d for _, d, _ in copies}:
            return                   # a table named a free page: what a copy of it holds is nobody's
        for c, old in zip(self.caches, before):
            block = c.block
            for s, d, n in copies:
                for i in (0, 1):
                    old[i][d, :, :n] = old[i][s, :, :n].clone()
                    m = -(-n // block)
                    old[2 + i][d, :, :m] = old[2 + i][s, :, :m].clone()
            for t, o in zip((c.k, c.v, c.k_scale, c.v_scale), old):
                assert torch.equal(t, o)

    def put(self):
        """The Python form's state to the device (after the test changed it)."""
        self.pool.refs.copy_(self.ints(self.ref.refs))
        self.pool.seq_lens.copy_(self.ints(self.ref.lens))
        self.pool.block_table.copy_(self.ints(self.ref.table))

    def free(self, rows):
        old = self.contents()
        self.ref.free(rows)
        dl.kv_free(self.pool, self.ints(rows))
        self.check(old, [])

    def reserve(self, rows, tokens):
        old = self.contents()
        want = self.ref.reserve(rows, tokens)
        assert dl.kv_reserve(self.pool, self.ints(rows), self.ints(tokens)).tolist() == want
        self.check(old, [])
        return want

    def fork(self, parents, children):
        old = self.contents()
        want, copies = self.ref.fork(parents, children)
        assert dl.kv_fork(self.pool, self.ints(parents), self.ints(children)).tolist() == want
        self.check(old, copies)
        return want

    def compact(self):
        old = self.contents()
        live, moves = self.ref.compact()
        assert dl.kv_compact(self.pool).tolist() == [live]
        self.check(old, [(s, d, self.ref.page) for s, d in moves])
        return live


def test_one_of_each(cuda_device):
    b = Both(cuda_device)
    assert b.reserve([0, 3], [40, 5]) == [1, 1]
    assert b.fork([0, 0, 3], [1, 2, 7]) == [1, 1, 1]
    assert b.ref.refs[0] == 3            # a shared page
    b.reserve([0, 1, 2, 3, 7], [1, 9, 16, 11, 0])
    b.free([0])
    b.free([3, 2])
    assert b.compact() == sum(c > 0 for c in b.ref.refs)
    b.free(list(range(8)))
    assert b.compact() == 0 and not any(b.ref.refs)


@pytest.mark.parametrize("seed", range(12))
def test_any_order_of_steps(cuda_device, seed):
    """Steps in any order with lists that name rows twice, out of range, empty and full ones, in pools
    that run out."""
    r = random.Random(seed)
    page = r.choice([8, 16, 64])
    b = Both(cuda_device, num_pages=r.choice([5, 23, 60]), page=page, rows=7, cols=r.choice([1, 4, 9]), layers=r.choice([0, 1, 3]),
             heads=r.choice([1, 3]), dim=r.choice([64, 128]), block=r.choice([1, 4, 8]), strided=seed % 2 == 1)
    some = lambda: [r.randint(-2, 8) for _ in range(r.randint(0, 7))]   # noqa: E731
    for _ in range(40):
        step = r.choice(["free", "reserve", "reserve", "fork", "fork", "compact"])
        if step == "free":
            b.free(some()[:2])
        elif step == "reserve":
            rows = some()
            b.reserve(rows, [r.choice([0, 1, 1, page, r.randint(0, 3 * page), -1, 2 ** 31 - 1]) for _ in rows])
        elif step == "fork":
            kids = some()
            b.fork([r.randint(-1, 7) for _ in kids], kids)
        else:
            b.compact()
    assert all(c >= 0 for c in b.ref.refs)


def test_empty_lists_and_full_lists(cuda_device):
    b = Both(cuda_device, rows=3)
    assert b.reserve([], []) == b.fork([], []) == []
    b.free([])
    assert b.reserve([2, 0, 1], [1, 2, 3]) == [1, 1, 1]
    with pytest.raises(dl.DLError, match="n=4"):
        dl.kv_free(b.pool, b.ints([0, 0, 0, 0]))


def test_pages_run_out(cuda_device):
    """Items are served in their order until the first that finds too few; those that need none still are."""
    b = Both(cuda_device, num_pages=5, page=8, rows=6, cols=9)
    assert b.reserve([0, 1, 2, 3], [17, 8, 16, 1]) == [1, 1, 0, 0]
    assert b.reserve([0, 1], [7, 0]) == [1, 1]
    assert b.reserve([2, 3], [9, 1]) == [0, 0]
    assert b.reserve([3], [1]) == [1]
    assert b.fork([3, 1, 0], [4, 5, 2]) == [0, 1, 1]       # row 3's page is begun, 1's and 0's are full
    b.free([0])
    assert b.ref.refs[:3] == [1, 1, 1]


@pytest.mark.parametrize("seed", range(4))
def test_contained_states(cuda_device, seed):
    """Tables, lengths and counts out of range: contained as documented."""
    r = random.Random(100 + seed)
    b = Both(cuda_device, num_pages=20, page=8, rows=8, cols=4)
    wild = [-1, 20, 2 ** 31 - 1, -2 ** 31]
    for row in range(8):
        b.ref.table[row] = [r.choice(wild + [r.randint(0, 19)] * 3) for _ in range(4)]
        b.ref.lens[row] = r.choice([-5, 0, 3, 8, 31, 32, 33, 2 ** 31 - 1, r.randint(1, 32)])
    b.ref.refs = [r.choice([-3, 0, 1, 2]) for _ in range(20)]
    b.put()
    b.reserve([0, 1, 2], [1, 1, 9])
    b.fork([3, 4, 5], [6, 7, 0])
    b.compact()
    b.free([5, 4, 4, 0])
    b.compact()


def test_alignment_of_the_lists(cuda_device):
    """refs that no 16-byte boundary begins, and lists that lie anywhere."""
    b = Both(cuda_device, num_pages=37)
    pool = torch.zeros(40, dtype=torch.int32, device=cuda_device)
    b.pool = dl.PagePool(b.caches, b.pool.block_table, b.pool.seq_lens, pool[1:38])
    b.reserve([0, 1], [50, 20])
    b.fork([0], [2])
    b.free([0])
    b.compact()
    assert pool[0] == 0 and not pool[38:].any()


def test_many_layers(cuda_device):
    """More caches than one launch takes."""
    b = Both(cuda_device, num_pages=12, page=8, rows=4, cols=3, layers=131, heads=1, block=8)
    b.reserve([0, 1], [13, 20])
    b.fork([0, 1], [2, 3])
    b.free([0, 1])
    b.compact()


def test_large_pool(cuda_device):
    """More pages than the planning CTA looks at in one round, most of them taken, and long rows."""
    n, page, rows, cols = 70001, 8, 40, 2500
    b = Both(cuda_device, num_pages=n, page=page, rows=rows, cols=cols, layers=1, heads=1, block=8)
    b.reserve(list(range(27)), [page * cols - i for i in range(27)])
    b.free(list(range(0, 27, 2)))
    b.compact()
    b.fork([1, 1, 3, 25], [0, 2, 4, 30])
    assert b.reserve([6, 8, 10], [20000, 20000, 19999]) == [1, 1, 1]
    b.free([1, 3, 0])
    b.compact()


def test_largest_rows(cuda_device):
    b = Both(cuda_device, num_pages=20000, page=8, rows=16384, cols=2, layers=0)
    rows = list(range(16384))
    random.Random(0).shuffle(rows)
    assert b.reserve(rows, [i % 9 for i in range(16384)])[:9] == [1] * 9
    b.free(rows[:8192])
    b.fork(rows[8192:], rows[:8192])
    b.compact()


def test_graph(cuda_device):
    """A beam step captured and replayed: the same as its calls, twice."""
    b, e = Both(cuda_device), Both(cuda_device)
    for x in (b, e):
        x.reserve([0, 1, 2], [20, 33, 7])
        x.fork([0, 1], [4, 5])
    ws = dl.Workspace(dl.pages_workspace_bytes(b.pool))
    par, kids, add = b.ints([0, 2]), b.ints([4, 5]), b.ints([3, 1])

    def step(pool):
        dl.kv_free(pool, kids)
        a = dl.kv_fork(pool, par, kids, workspace=ws)
        c = dl.kv_reserve(pool, kids, add, workspace=ws)
        return a, c, dl.kv_compact(pool, workspace=ws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(b.pool)
    for _ in range(2):
        graph.replay()
        want = step(e.pool)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        for n in ("refs", "seq_lens", "block_table"):
            assert torch.equal(getattr(b.pool, n), getattr(e.pool, n))
        for c, d in zip(b.contents(), e.contents()):
            assert all(torch.equal(x, y) for x, y in zip(c, d))
    assert not ws.tensor[:dl.WORKSPACE_ZERO_BYTES].any()


def test_other_stream(cuda_device):
    b = Both(cuda_device)
    side = torch.cuda.Stream()
    b.reserve([0], [20])
    rows, kids = b.ints([0]), b.ints([1])
    side.wait_stream(torch.cuda.current_stream())
    done = dl.kv_fork(b.pool, rows, kids, stream=side)
    live = dl.kv_compact(b.pool, stream=side.cuda_stream)
    side.synchronize()
    assert done.tolist() == [1] and live.tolist() == [3]
    dl.kv_free(b.pool, kids, stream=side)
    side.synchronize()
    assert b.pool.refs.tolist()[:3] == [1, 1, 0]


def test_refusals(cuda_device):
    b = Both(cuda_device)
    x = b.ints([0, 1])
    for f, match in ((lambda: dl.kv_free(b.pool, x.long()), "rows"), (lambda: dl.kv_free(b.pool, x.cpu()), "rows"),
                     (lambda: dl.kv_reserve(b.pool, x, x[:1]), r"\[n\]"), (lambda: dl.kv_fork(b.pool, x, x.float()), "children"),
                     (lambda: dl.kv_fork(b.pool, x, x, out_done=x[:1]), "out_done"),
                     (lambda: dl.kv_compact(b.pool, out_live=x), "out_live"),
                     (lambda: dl.PagePool(b.caches, b.pool.block_table, b.pool.seq_lens, x), "one shape"),
                     (lambda: dl.PagePool(b.caches, b.pool.block_table, x, b.pool.refs), "rows"),
                     (lambda: dl.PagePool([], b.pool.block_table, b.pool.seq_lens, b.pool.refs), "page_size")):
        with pytest.raises(ValueError, match=match):
            f()
    with pytest.raises(TypeError, match="children"):
        dl.kv_fork(b.pool, x, [0, 1])
    with pytest.raises(dl.DLError, match="workspace"):
        dl.kv_compact(b.pool, workspace=dl.Workspace(1000))
