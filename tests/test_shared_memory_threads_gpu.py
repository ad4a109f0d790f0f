"""Threads that launch one kernel with more and with less shared memory, each on its own stream, outputs and
workspace: no call takes from another what it has asked for.

The threads call the library from C, so that nothing but the library's own work lies between two calls.
"""
import ctypes
import subprocess

import pytest
import torch

import weight_streaming_skinny_gb300 as dl
from weight_streaming_skinny_gb300 import build

pytestmark = pytest.mark.gpu

CALLS = 4000

CODE = """
#include <pthread.h>
#include <stddef.h>
#include "dl_linear.h"

typedef struct {
    int (*call)(const void* const*, const int*, void*, size_t, void*);
    const void* p[8];
    int n[4];
    void* ws;
    size_t bytes;
    void* stream;
    int calls, status, done;
} job;

static pthread_barrier_t start;

static void* run(void* arg) {
    job* j = arg;
    pthread_barrier_wait(&start);
    for (; j->done < j->calls && !j->status; ++j->done) j->status = j->call(j->p, j->n, j->ws, j->bytes, j->stream);
    return NULL;
}
void two(job* a, job* b) {
    pthread_t t;
    pthread_barrier_init(&start, NULL, 2);
    pthread_create(&t, NULL, run, a);
    run(b);
    pthread_join(t, NULL);
    pthread_barrier_destroy(&start);
}
static dl_status (*norm_fn)(const dl_rows*, const dl_norm*, const dl_rows*, int, int, float, const dl_rows*, float,
                            const dl_norm*, const dl_rows*, const dl_rows*, int, int, void*);
static dl_status (*adapters_fn)(const dl_adapters*, const dl_rows*, const int*, const dl_rows*, const dl_rows*,
                                const dl_rows*, int, void*, size_t, void*);
static dl_status (*reserve_fn)(const dl_kv_pages*, const int*, const int*, int*, int, void*, size_t, void*);
void bind(void* norm, void* adapters, void* reserve) {
    *(void**)&norm_fn = norm;
    *(void**)&adapters_fn = adapters;
    *(void**)&reserve_fn = reserve;
}
int norm(const void* const* p, const int* n, void* ws, size_t bytes, void* stream) {
    (void)ws, (void)bytes;
    return norm_fn(p[0], NULL, NULL, DL_GATE_NONE, DL_GATE_PLAIN, 1.f, p[1], 1.f, p[2], p[3], p[4], n[0], n[1], stream);
}
int adapters(const void* const* p, const int* n, void* ws, size_t bytes, void* stream) {
    return adapters_fn(p[0], p[1], p[2], NULL, p[3], NULL, n[0], ws, bytes, stream);
}
int reserve(const void* const* p, const int* n, void* ws, size_t bytes, void* stream) {
    return reserve_fn(p[0], p[1], p[2], (int*)p[3], n[0], ws, bytes, stream);
}
"""

vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t


class Job(ctypes.Structure):
    _fields_ = [("call", vp), ("p", vp * 8), ("n", i * 4), ("ws", vp), ("bytes", sz), ("stream", vp), ("calls", i), ("status", i),
                ("done", i)]


class Rows(ctypes.Structure):
    _fields_ = [("data", vp), ("stride", ctypes.c_longlong), ("dtype", i)]


def rows(t):
    return Rows(t.data_ptr(), t.stride(0), int(t.dtype == torch.float32))


class Call:
    """One call's arguments: structures and tensors in `p`, sizes in `n`; `out` is what it writes."""

    def __init__(self, name, p, n, out, ws=None):
        self.name, self.p, self.n, self.out, self.ws = name, p, n, out, ws

    def job(self, lib, stream, calls):
        at = [t.data_ptr() if isinstance(t, torch.Tensor) else ctypes.addressof(t) for t in self.p]
        fn = ctypes.cast(getattr(lib, self.name), vp)
        return Job(fn, (vp * 8)(*at), (i * 4)(*self.n), None if self.ws is None else self.ws.addr,
                   0 if self.ws is None else self.ws.nbytes, stream.cuda_stream, calls, 0, 0)


def adapters(dev, num, rank, tokens, in_runs):
    g = torch.Generator(device=dev).manual_seed(rank)
    rand = lambda *s: (torch.randn(*s, device=dev, generator=g) / 8).bfloat16()   # noqa: E731
    a, b = (torch.zeros(s, dtype=torch.bfloat16, device=dev) for s in ((num, rank, 64), (num, 64, rank)))
    a[:3], b[:3] = rand(3, rank, 64), rand(3, 64, rank)
    index = torch.arange(tokens, device=dev, dtype=torch.int32)
    ad, x, out = dl.Adapters(a, b), rand(tokens, 64), torch.zeros(tokens, 64, dtype=torch.bfloat16, device=dev)
    index = index * 3 // tokens if in_runs else index % 3
    c = Call("adapters", [ad._struct, rows(x), index, rows(out)], [tokens], out, dl.Workspace(dl.adapters_workspace_bytes(tokens, ad)))
    c.keep = ad, x
    return c


def norm(dev, dim):
    g = torch.Generator(device=dev).manual_seed(dim)
    h = torch.randn(700, dim, device=dev, generator=g)
    y, pre, r, x = h.bfloat16(), dl.Norm(), torch.zeros_like(h), torch.zeros_like(h, dtype=torch.bfloat16)
    c = Call("norm", [rows(y), rows(h), pre._struct, rows(r), rows(x)], [700, dim], x)
    c.keep = y, h, pre, r
    return c


def pool(dev, n):
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)   # noqa: E731
    p = dl.PagePool([], zeros(n, 1) - 1, zeros(n), zeros(8), page_size=8)
    done = zeros(4) + 7
    c = Call("reserve", [p._struct, torch.arange(4, device=dev, dtype=torch.int32), zeros(4), done], [4], done,
             dl.Workspace(dl.pages_workspace_bytes(p)))
    c.keep = p
    return c


@pytest.mark.parametrize("what", ["tiles", "sort", "norm", "pages"])
def test_two_threads(cuda_device, tmp_path, what):
    dev = cuda_device
    src, so = tmp_path / "two.c", tmp_path / "two.so"
    src.write_text(CODE)
    subprocess.run(["gcc", "-O2", "-std=gnu11", "-shared", "-fPIC", "-pthread", "-I", build.INCLUDE, "-o", str(so), str(src)],
                   check=True)
    lib, own = ctypes.CDLL(str(so)), dl.load()
    lib.bind(*[ctypes.cast(f, vp) for f in (own.dl_block_norm, own.dl_linear_adapters, own.dl_kv_reserve)])
    calls = {"tiles": lambda: (adapters(dev, 3, 128, 300, True), adapters(dev, 3, 16, 300, True)),
             "sort": lambda: (adapters(dev, 16384, 8, 400, False), adapters(dev, 13000, 8, 300, False)),
             "norm": lambda: (norm(dev, 8192), norm(dev, 5120)),
             "pages": lambda: (pool(dev, 16384), pool(dev, 13000))}[what]()
    streams = [torch.cuda.Stream(dev) for _ in calls]
    torch.cuda.synchronize(dev)
    want = []
    for n in (1, CALLS):                 # one after the other, then both at the same time
        jobs = [c.job(lib, s, n) for c, s in zip(calls, streams)]
        if n == 1:
            for j in jobs:
                none = Job(j.call, calls=0)
                lib.two(ctypes.byref(j), ctypes.byref(none))
        else:
            lib.two(*map(ctypes.byref, jobs))
        torch.cuda.synchronize(dev)
        assert [(j.status, j.done) for j in jobs] == [(0, n)] * 2
        want.append([c.out.clone() for c in calls])
    assert all(torch.equal(a, b) for a, b in zip(*want))
    assert dl.device_status() == 0
