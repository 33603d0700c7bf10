"""Host code of the operators around the layer under AddressSanitizer (no GPU):
workspace sizes of many problems and the refusals of every entry point."""

import os
import subprocess
import sys

from test_host_asan import ROOT, asan_lib  # noqa: F401

DRIVER = r"""
import ctypes, random, sys
lib = ctypes.CDLL(sys.argv[1])
class P(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("d", "E", "k", "de", "dt")]
rng, n, calls = random.Random(3), ctypes.c_size_t(0), 0
for _ in range(200):
    E = rng.randint(1, 256)
    p = P(rng.randint(1, 70000), 64 * rng.randint(1, 130), E, rng.randint(1, min(E, 8)), 64 * rng.randint(1, 130),
          rng.randint(0, 1))
    for st in range(-1, 7):
        r = lib.moex_workspace_size(ctypes.byref(p), st, ctypes.byref(n))
        assert r == (0 if 0 <= st <= 4 else 1) and (r or n.value > 0), (st, r)
        calls += 1
vp = ctypes.c_void_p
at = lambda i: vp((i + 1) << 40)
p = ctypes.byref(P(64, 128, 8, 2, 256, 1))
f = ctypes.c_float
small = ctypes.c_size_t(1)
a = [at(i) for i in range(16)]
for got, want in (
    (lib.moex_add_rmsnorm(p, a[0], a[1], a[2], f(float("nan")), a[3], a[4], a[5], a[6], a[7], None), 1),
    (lib.moex_add_rmsnorm(p, a[0], a[1], a[2], f(0), a[0], a[4], a[5], a[6], a[7], None), 1),
    (lib.moex_add_rmsnorm_backward(p, *a[:8], small, None), 3),
    (lib.moex_quantize_rows(p, a[0], a[0], a[1], None), 1),
    (lib.moex_balance_loss(p, a[0], a[1], a[2], f(1), a[3], a[4], a[5], a[6], a[7], small, None), 3),
    (lib.moex_backward_balanced(p, *a[:6], f(1), *a[6:15], small, None), 3),
    (lib.moex_quantize_experts(p, *a[:5], None, None), 1),
    (lib.moex_grouped_ffn_fp8(p, *a[:10], small, None), 3),
    (lib.moex_forward_fp8(p, *a[:11], small, None), 3),
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
