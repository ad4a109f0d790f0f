"""Launches near the shared memory that a kernel has without asking for more: 48 KB, its own static part counted in.

Each case in a process of its own: a larger call before it would have asked already.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INTS = 48 * 1024 // 4                    # the planning and sorting kernels' dynamic part is of integers

SCRIPT = """
import sys, torch
import weight_streaming_skinny_gb300 as dl
what, n = sys.argv[1], int(sys.argv[2])
dev = torch.device("cuda:0")
ints = lambda t: t.int().to(dev)
if what in ("reserve", "fork"):          # an integer a row
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    pool = dl.PagePool([], zeros(n, 2) - 1, zeros(n), zeros(2 * n), page_size=8)
    half = torch.arange(n // 2)
    if what == "reserve":
        done = dl.kv_reserve(pool, ints(half), ints(torch.full((n // 2,), 11)))
        assert bool(done.all()) and int(pool.refs.sum()) == 2 * (n // 2) and pool.seq_lens[:3].tolist() == [11] * 3
    else:
        pool.seq_lens[:n // 2] = 8
        pool.block_table[:n // 2, 0] = ints(half)
        pool.refs[:n // 2] = 1
        done = dl.kv_fork(pool, ints(half), ints(half + n // 2))
        assert bool(done.all()) and pool.refs[:n // 2].eq(2).all() and pool.seq_lens[n // 2:n // 2 * 2].eq(8).all()
        assert torch.equal(pool.block_table[n // 2:n // 2 * 2, 0], ints(half))
else:                                    # an integer an adapter, one more, and, of few tokens, one more than tokens
    T = int(what)
    num = n - 1 - (T + 1 if T <= 8192 else 0)
    a = torch.zeros(num, 8, 16, dtype=torch.bfloat16, device=dev)
    b = torch.ones(num, 16, 8, dtype=torch.bfloat16, device=dev)
    a[:, 0, 0] = torch.arange(num, device=dev) % 128
    index = torch.arange(T) * 37 % num
    x = torch.ones(T, 16, dtype=torch.bfloat16, device=dev)
    out = dl.linear_adapters(x, dl.Adapters(a, b), ints(index))
    assert torch.equal(out.float().cpu(), (index % 128).float()[:, None].expand(T, 16))
torch.cuda.synchronize()
"""


@pytest.mark.parametrize("what,n", [("reserve", INTS - 63), ("reserve", INTS), ("reserve", INTS + 1), ("fork", INTS),
                                    ("300", INTS - 63), ("300", INTS), ("9000", INTS)])
def test_a_first_call(what, n):
    r = subprocess.run([sys.executable, "-c", SCRIPT, what, str(n)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
