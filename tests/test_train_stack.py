"""The list calls on a thread with a small stack (no GPU: each call is refused after its checks)."""

import subprocess
import sys

import pytest

DRIVER = r"""
import ctypes, sys, threading
lib = ctypes.CDLL(sys.argv[1])
class T(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "master", "m", "v", "ms", "vs")] + [
        ("n", ctypes.c_int64), ("pd", ctypes.c_int32), ("gd", ctypes.c_int32), ("lf", ctypes.c_double), ("wd", ctypes.c_double)]
class O(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "b1", "b2", "eps")] + [("seed", ctypes.c_uint32)]
vp, d, small = ctypes.c_void_p, ctypes.c_double, ctypes.c_size_t(1)
at = lambda i: vp((i + 1) << 34)
o = ctypes.byref(O(1e-3, .9, .99, 1e-8, 1))
def entries(count):
    arr = (T * count)()
    for i in range(count):
        b = 10 * i
        arr[i] = T(*(at(b + j).value for j in range(7)), 100, 1, 1, 1.0, 0.1)
    return arr
calls = []
for count in (1, 16, 17, 18, 200, 1024):
    arr, twice = entries(count), entries(count)
    twice[count - 1].v = twice[0].m  # two outputs in one place, found only when all are known
    calls += [(lib.moet_adamw, (twice, count, o, at(99999), None, None, None), 1),
              (lib.moet_adamw_clipped, (twice, count, o, at(99999), None, d(1), at(99998), None, at(99997), small, None), 1),
              (lib.moet_adamw_clipped, (arr, count, o, at(99999), None, d(1), at(99998), at(99996), at(99997), small, None), 3),
              (lib.moet_grad_norm, (arr, count, d(1), at(99999), at(99998), at(99997), small, None), 3)]
got = []
def run():
    for f, a, want in calls:
        got.append((f(*a), want))
threading.stack_size(int(sys.argv[2]))
t = threading.Thread(target=run)
t.start()
t.join()
assert len(got) == len(calls) and all(a == b for a, b in got), got
print("ok")
"""


@pytest.mark.parametrize("stack", [96 << 10, 8 << 20])
def test_long_lists_need_little_stack(libmoe_path, stack):
    r = subprocess.run([sys.executable, "-c", DRIVER, libmoe_path, str(stack)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout + r.stderr[-2000:])
