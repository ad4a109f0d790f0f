"""Threads that share a workspace: a call's kernels hand each other results through it, so the launches of two
calls on one workspace must not mix, on whatever thread they are made (no GPU needed: the library's calls are
stand-ins that take a while, as they do where the driver's queue is full).
"""
import contextlib
import threading
import time
from types import SimpleNamespace

import pytest
import torch

import weight_streaming_skinny_gb300 as dl

DEV = torch.device("cpu")


class Library:
    """Stands in for the library and for the C module: counts the threads that are inside a call at once, and the
    workspaces' addresses that were passed."""

    def __init__(self):
        self.lock, self.inside, self.most, self.meet = threading.Lock(), 0, 0, None

    def call(self, *args):
        with self.lock:
            self.inside += 1
            self.most = max(self.most, self.inside)
        if self.meet is not None:
            self.meet.wait()             # (raises if the other call cannot come in)
        time.sleep(0.01)
        with self.lock:
            self.inside -= 1
        return 0

    def __getattr__(self, name):
        if not name.startswith("dl_"):
            raise AttributeError(name)
        return (lambda *args: 4096) if name.endswith("_bytes") else self.call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(dl, "load", lambda: lib)
    monkeypatch.setattr(dl, "_native", {n: lib.call for n in ("attention", "adapters", "pages")})
    monkeypatch.setattr(dl, "_default_ws", {})
    monkeypatch.setattr(dl, "_outgrown", [])
    for n in ("_need", "_explain_attention", "_explain_adapters"):
        monkeypatch.setattr(dl, n, lambda *a, **k: None)
    monkeypatch.setattr(dl, "_layer_struct", lambda layer: dl._Layer())
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "synchronize", lambda d=None: time.sleep(0.01))
    return lib


def calls():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)   # noqa: E731
    ints = torch.zeros(2, dtype=torch.int32)
    codes, scales = torch.zeros(128, 128, dtype=torch.uint8), torch.ones(1, 1)
    ad = SimpleNamespace(device=DEV, num=2, rank=8, parts=[8], N=8, _args=())
    cache = SimpleNamespace(device=DEV, kv_heads=1, head_dim=64, _args=())
    pool = SimpleNamespace(device=DEV, num_pages=4, rows=2, _args=())
    out = torch.empty(2, dtype=torch.int32)
    return {
        "linear_bf16": lambda **k: dl.linear_bf16(bf(1, 8), bf(8, 8), **k),
        "linear_swiglu": lambda **k: dl.linear_swiglu(bf(1, 8), bf(16, 8), **k),
        "linear_argmax": lambda **k: dl.linear_argmax(bf(1, 8), bf(8, 8), **k),
        "linear_fp8_block128": lambda **k: dl.linear_fp8_block128(bf(1, 128), codes, scales, **k),
        "attention_paged": lambda **k: dl.attention_paged(bf(2, 1, 64), cache, ints[None], ints, ints, max_q=1, **k),
        "linear_adapters": lambda **k: dl.linear_adapters(bf(2, 8), ad, ints, **k),
        "kv_reserve": lambda **k: dl.kv_reserve(pool, ints, ints, out_done=out, **k),
        "kv_fork": lambda **k: dl.kv_fork(pool, ints, ints, out_done=out, **k),
        "kv_compact": lambda **k: dl.kv_compact(pool, out_live=out[:1], **k),
    }


def threads(*fns):
    """Run them at the same time; raise what the first one raised."""
    errors, start = [], threading.Barrier(len(fns))

    def run(fn):
        try:
            start.wait()
            fn()
        except BaseException as e:       # noqa: BLE001
            errors.append(e)

    all_ = [threading.Thread(target=run, args=(f,)) for f in fns]
    for t in all_:
        t.start()
    for t in all_:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("name", list(calls()))
def test_calls_on_one_default_workspace(lib, name):
    call = calls()[name]
    threads(*[lambda: [call(stream=7) for _ in range(3)]] * 3)
    assert lib.most == 1


@pytest.mark.parametrize("name", list(calls()))
def test_different_calls_on_one_default_workspace(lib, name):
    one, other = calls()[name], calls()["linear_adapters"]
    threads(lambda: [one(stream=7) for _ in range(3)], lambda: [other(stream=7) for _ in range(3)])
    assert lib.most == 1


@pytest.mark.parametrize("name", list(calls()))
def test_calls_on_two_workspaces(lib, name):
    """Each is inside while the other one is."""
    call = calls()[name]
    lib.meet = threading.Barrier(2, timeout=20)
    threads(lambda: call(stream=7), lambda: call(stream=8))
    assert lib.most == 2


@pytest.mark.parametrize("name", list(calls()))
def test_calls_on_one_workspace_of_the_caller(lib, name):
    call, ws = calls()[name], dl.Workspace(4096, DEV)
    threads(*[lambda: [call(workspace=ws, stream=s) for s in (7, 8)]] * 3)
    assert lib.most == 1


def test_a_workspace_over_other_memory(lib):
    """One that is made without its constructor, from a part of a larger buffer."""
    ws = dl.Workspace.__new__(dl.Workspace)
    ws.nbytes, ws.tensor = 4096, torch.zeros(4096, dtype=torch.uint8)
    call = calls()["linear_bf16"]
    threads(*[lambda: call(workspace=ws, stream=7)] * 3)
    assert lib.most == 1


def test_streams_of_layers_on_one_workspace(lib):
    ws = dl.Workspace(4096, DEV)
    layers = [SimpleNamespace(x=torch.zeros(1, 8))] * 2
    threads(*[lambda: [dl.decode_stream(layers, ws, stream=7) for _ in range(3)]] * 3)
    assert lib.most == 1


def test_a_call_within_a_call(lib):
    """What runs in the middle of a call on the same thread (a finaliser, a signal's handler) may call too."""
    ws = dl.Workspace(4096, DEV)
    inner = calls()["kv_fork"]
    dl._native["adapters"] = lambda *a: inner(workspace=ws, stream=7) is None
    t = threading.Thread(target=lambda: calls()["linear_adapters"](workspace=ws, stream=7), daemon=True)
    t.start()
    t.join(20)
    assert not t.is_alive()


def test_one_default_workspace(lib):
    """First calls of many threads make one; a larger one leaves the smaller one to who has it."""
    got, lock = [], threading.Lock()

    def take(need):
        ws = dl._workspace(None, need, DEV, 7)
        with lock:
            got.append((need, ws))

    threads(*[lambda n=n: take(n) for n in (4096, 4096, 1 << 20, 4096, 8192, 1 << 20)])
    kept = list(dl._default_ws.values()) + dl._outgrown
    assert all(ws.nbytes >= n and any(ws is k for k in kept) for n, ws in got)
    assert dl._default_ws[(None, 7)].nbytes == 1 << 20
    assert len(kept) == len({k.nbytes for k in kept})
