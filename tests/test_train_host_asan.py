"""Host code of what trains the layer's surroundings under AddressSanitizer (no GPU):
workspace sizes of many problems, and refusals of every entry point, of full lists too."""

import os
import subprocess
import sys

from test_host_asan import ROOT, asan_lib  # noqa: F401

DRIVER = r"""
import ctypes, random, sys
lib = ctypes.CDLL(sys.argv[1])
class P(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("d", "E", "k", "de", "dt")]
class T(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "master", "m", "v", "ms", "vs")] + [
        ("n", ctypes.c_int64), ("pd", ctypes.c_int32), ("gd", ctypes.c_int32), ("lf", ctypes.c_double), ("wd", ctypes.c_double)]
class O(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "b1", "b2", "eps")] + [("seed", ctypes.c_uint32)]
rng, n, calls = random.Random(4), ctypes.c_size_t(0), 0
for _ in range(300):
    E = rng.randint(1, 256)
    p = P(rng.randint(1, 70000), 64 * rng.randint(1, 130), E, rng.randint(1, min(E, 8)), 64 * rng.randint(1, 130),
          rng.randint(0, 1))
    for st in range(-1, 5):
        r = lib.moet_workspace_size(ctypes.byref(p), st, ctypes.byref(n))
        assert r == (0 if 0 <= st <= 2 else 1) and (r or n.value > 0), (st, r)
        calls += 1
vp = ctypes.c_void_p
at = lambda i: vp((i + 1) << 34)
p = ctypes.byref(P(64, 128, 8, 2, 256, 1))
small = ctypes.c_size_t(1)
a = [at(i) for i in range(16)]
libc = ctypes.CDLL(None)
libc.malloc.restype = vp
libc.malloc.argtypes = [ctypes.c_size_t]
def full(count, last):
    # entries in malloc'ed memory of exactly their size: a read past them lands in a redzone
    raw = libc.malloc(count * ctypes.sizeof(T))
    arr = ctypes.cast(raw, ctypes.POINTER(T))
    for i in range(count):
        b = 10 * i
        arr[i] = T(at(b).value, at(b + 1).value, at(b + 2).value, at(b + 3).value, at(b + 4).value, None, None, 100, 1, 1, 1.0, 0.1)
    arr[count - 1].param = last
    return arr
o = ctypes.byref(O(1e-3, .9, .99, 1e-8, 1))
for got, want in (
    (lib.moet_dispatch(p, *a[:9], small, None), 3),
    (lib.moet_dispatch_backward(p, *a[:5], a[0], a[6], None), 1),
    (lib.moet_combine(p, *a[:4], a[0], None), 1),
    (lib.moet_combine_backward(p, *a[:4], a[0], a[5], None), 1),
    (lib.moet_gate_backward(p, *a[:4], a[0], None), 1),
    (lib.moet_linear(p, a[0], a[1], a[2], 1, a[3], a[4], a[5], a[6], small, None), 3),
    (lib.moet_linear_backward(p, a[0], a[1], a[2], 1, a[3], a[4], a[5], a[6], a[7], small, None), 3),
    (lib.moet_adamw(full(1, None), 1, o, at(99999), None, None, None), 1),
    (lib.moet_adamw(full(1024, at(1).value), 1024, o, at(99999), None, None, None), 1),
    (lib.moet_adamw_clipped(full(1024, at(1).value), 1024, o, at(99999), None, ctypes.c_double(1), at(99998), None, at(99997), small, None), 1),
    (lib.moet_grad_norm(full(1024, None), 1024, ctypes.c_double(1), at(99999), at(99998), at(99997), small, None), 3),
):
    assert got == want, (got, want)
    calls += 1
print("ok", calls)
"""


def test_host_paths_make_no_invalid_access(asan_lib):  # noqa: F811
    lib, rt = asan_lib
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0")
    r = subprocess.run([sys.executable, "-c", DRIVER, lib], env=env, capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr[-4000:]
