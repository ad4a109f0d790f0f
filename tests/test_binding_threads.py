"""The cache's calls let other Python threads run while the library is in a call (no GPU needed).

A launch waits where the driver's queue is full; a thread that feeds the GPU must be able to run then.
"""
import subprocess
import sys
import textwrap

import pytest

from weight_streaming_skinny_gb300 import build

SLOW = """
#include <unistd.h>
int slow(void) { usleep(400000); return 0; }
int device(int* d) { *d = 0; return 0; }
"""

SCRIPT = """
import ctypes, importlib.util, sys, threading, time
path, lib, name = sys.argv[1:]
spec = importlib.util.spec_from_file_location("_binding", path)
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
lib = ctypes.CDLL(lib)
at = lambda f: ctypes.cast(f, ctypes.c_void_p).value
bf16, i32, f32 = object(), object(), object()

class T:                      # what the binding asks of a tensor
    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, shape
    def stride(self):
        s, n = [], 1
        for d in reversed(self.shape):
            s.insert(0, n)
            n *= d
        return tuple(s)
    def get_device(self): return 0
    def is_contiguous(self): return True
    def data_ptr(self): return 4096

b.bind(T, bf16, i32, f32, lambda d: 0, at(lib.device), at(lib.slow), at(lib.slow), at(lib.slow))
q, kv, seq = T(bf16, 2, 4, 128), T(bf16, 2, 2, 128), (T(i32, 1, 3), T(i32, 1), T(i32, 2))
call = {"append": lambda: b.append(4096, 0, 2, 128, q, kv, kv, *seq, 2, None, None, None, q, 0),
        "attention": lambda: b.attention(4096, 0, 2, 128, q, *seq, 2, 0.1, q, None, 4096, 1 << 20, 0),
        "verify": lambda: b.verify(0, T(i32, 2, 3), T(f32, 2, 4, 9), T(f32, 2, 3), T(f32, 2), None, None, T(i32, 2, 4),
                                   T(i32, 2), 0)}[name]
turns, stop = 0, False
def other():
    global turns
    while not stop:
        time.sleep(0.01)
        turns += 1
t = threading.Thread(target=other)
t.start()
time.sleep(0.1)
before = turns
status = call()
during = turns - before
stop = True
t.join()
print(status, during)
"""


@pytest.mark.parametrize("name", ["append", "attention", "verify"])
def test_other_threads_run_during_a_call(tmp_path, name):
    build.build()
    src, lib = tmp_path / "slow.c", tmp_path / "slow.so"
    src.write_text(SLOW)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    script = tmp_path / "run.py"
    script.write_text(textwrap.dedent(SCRIPT))
    r = subprocess.run([sys.executable, str(script), build.BINDING, str(lib), name], capture_output=True, text=True,
                       timeout=60)
    assert r.returncode == 0, r.stderr
    status, during = map(int, r.stdout.split())
    assert status == 0
    assert during >= 5          # of 40 turns that fit into the 0.4 s
