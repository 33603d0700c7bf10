"""The dense projection and its gradients on the GPU, against float64.

Bounds. A sum of K products of bfloat16 values (exact in float32) is off by at most
(K + 40) 2^-24 of the sum of magnitudes: K additions in any order, and those of partial
sums, bias and residual. GELU and SiLU have slopes of at most 1.13 and add 2^-20 of the
argument (hardware exponential and reciprocal, each within 2^-22). A slope is off by at
most 2^-17: 1 - s of a sigmoid is off by 2^-23, times u z' of at most 35 where s is not
yet 1. dU is rounded to bfloat16, half a step, before it is multiplied, and each result
once more.
"""

import numpy as np
import pytest
import torch

from ext_helpers import HALF, assert_within, randn
from gpu_helpers import U32, announce, f64, needs_gpu
from oracle import train_ops as to
from test_gpu_canary import Guarded

pytestmark = [pytest.mark.gpu, needs_gpu]

BF = torch.bfloat16
ACTS = ["none", "gelu", "silu", "relu"]
H = HALF[BF]


def code(moe, act):
    return {"none": moe.MOET_ACT_NONE, "gelu": moe.MOET_ACT_GELU, "silu": moe.MOET_ACT_SILU, "relu": moe.MOET_ACT_RELU}[act]


class Linear:
    def __init__(self, moe, T, K, N, seed, guarded=False):
        self.moe, self.p, self.T, self.K, self.N = moe, moe.make_problem(T, K, 1, 1, N, BF), T, K, N
        self.x, self.W = randn((T, K), 1.0, BF, seed), randn((K, N), K ** -0.5, BF, seed + 1)
        self.bias, self.res, self.dy = randn((N,), 0.5, BF, seed + 2), randn((T, N), 1.0, BF, seed + 3), randn((T, N), 1.0, BF, seed + 4)
        make = (lambda s, t=BF: Guarded(s, t)) if guarded else (lambda s, t=BF: torch.full(s, 77, dtype=t, device="cuda"))
        self.out = {"u": make((T, N)), "y": make((T, N)), "dx": make((T, K)), "dW": make((K, N)), "db": make((N,)),
                    "ws": make((moe.moet_workspace_size(self.p, moe.MOET_STAGE_LINEAR),), torch.uint8),
                    "wsb": make((moe.moet_workspace_size(self.p, moe.MOET_STAGE_LINEAR_BACKWARD),), torch.uint8)}
        self.o = {n: v.t if guarded else v for n, v in self.out.items()}

    def forward(self, act, bias, residual, keep, stream=None):
        self.moe.moet_linear(self.p, self.x, self.W, self.bias if bias else None, code(self.moe, act),
                             self.res if residual else None, self.o["u"] if keep else None, self.o["y"], self.o["ws"], stream)

    def backward(self, act, stream=None):
        o = self.o
        self.moe.moet_linear_backward(self.p, self.x, self.W, o["u"], code(self.moe, act), self.dy, o["dx"], o["dW"], o["db"],
                                      o["wsb"], stream)

    def check_forward(self, act, bias, residual, keep):
        torch.cuda.synchronize()
        x, W = f64(self.x), f64(self.W)
        b = f64(self.bias) if bias else 0.0
        u = x @ W + b
        eu = (self.K + 40) * U32 * (np.abs(x) @ np.abs(W) + np.abs(b))
        if keep:
            assert_within("u", f64(self.o["u"]), u, eu + H * (np.abs(u) + eu))
        r = f64(self.res) if residual else 0.0
        y = to.act(u, act) + r
        ey = 1.13 * eu + (2.0 ** -20 * np.abs(u) if act in ("gelu", "silu") else 0.0) + 4 * U32 * (np.abs(u) + np.abs(r))
        assert_within("y", f64(self.o["y"]), y, ey + H * (np.abs(y) + ey))

    def check_backward(self, act):
        torch.cuda.synchronize()
        x, W, dy, u = f64(self.x), f64(self.W), f64(self.dy), f64(self.o["u"])
        du = dy * to.act_slope(u, act)
        es = 2.0 ** -17 * np.abs(dy) if act in ("gelu", "silu") else 0.0 * dy
        ed = es + (H * (np.abs(du) + es) if act != "none" else 0.0)
        aW, ax = np.abs(W), np.abs(x)
        dx = du @ W.T
        e = ed @ aW.T + (self.N + 40) * U32 * (np.abs(du) @ aW.T)
        assert_within("dx", f64(self.o["dx"]), dx, e + H * (np.abs(dx) + e))
        dW = x.T @ du
        e = ax.T @ ed + (self.T + 40) * U32 * (ax.T @ np.abs(du))
        assert_within("dW", f64(self.o["dW"]), dW, e + H * (np.abs(dW) + e))
        db = du.sum(0)
        e = es.sum(0) + (self.T + 40) * U32 * np.abs(du).sum(0)
        assert_within("db", f64(self.o["db"]), db, e + H * (np.abs(db) + e))


SHAPES = [(1, 64, 64), (1, 2048, 192), (2, 192, 1088), (31, 576, 320), (33, 320, 64), (64, 64, 2048), (100, 1024, 448),
          (129, 256, 704), (257, 704, 576), (600, 512, 320), (777, 320, 448)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_against_float64(moe, T, K, N, act):
    announce(f"linear T={T} K={K} N={N} {act}")
    c = Linear(moe, T, K, N, 1)
    for bias, residual, keep in ((True, True, True), (False, False, False), (True, False, True), (False, True, True)):
        c.forward(act, bias, residual, keep)
        c.check_forward(act, bias, residual, keep)
    c.backward(act)
    c.check_backward(act)


@pytest.mark.parametrize("tile,splits", [(0, 1), (0, 2), (1, 1), (1, 4), (2, 1), (2, 4)])
@pytest.mark.parametrize("T,K,N", [(300, 1280, 576), (70, 1088, 1088)])
def test_every_tile_and_cut(moe, monkeypatch, T, K, N, tile, splits):
    """Each tile and cut at shapes that end inside tiles, and steps along K that do not divide."""
    announce(f"linear tile={tile} splits={splits} T={T} K={K} N={N}")
    monkeypatch.setenv("MOE_LINEAR_TILE", str(tile))
    monkeypatch.setenv("MOE_LINEAR_SPLITS", str(splits))
    c = Linear(moe, T, K, N, 2)
    c.forward("gelu", True, True, True)
    c.check_forward("gelu", True, True, True)
    c.backward("gelu")
    c.check_backward("gelu")


def test_persistent_tiles(moe, monkeypatch):
    """More tiles than workgroups: results leave while the next tile's operands come in."""
    announce("linear rounds of tiles")
    for tile, (T, K, N) in ((0, (4352, 128, 4416)), (1, (4352, 192, 2240))):
        monkeypatch.setenv("MOE_LINEAR_TILE", str(tile))
        c = Linear(moe, T, K, N, 3)
        c.forward("silu", True, True, True)
        c.check_forward("silu", True, True, True)


def test_only_outputs_are_written(moe):
    for T, K, N in ((5, 320, 448), (300, 448, 320)):
        announce(f"linear guarded T={T}")
        c = Linear(moe, T, K, N, 4, guarded=True)
        inputs = [c.x, c.W, c.bias, c.res, c.dy]
        before = [t.clone() for t in inputs]
        c.forward("gelu", True, True, True)
        c.backward("gelu")
        c.check_backward("gelu")
        assert all(g.intact() for g in c.out.values())
        assert all(torch.equal(a, b) for a, b in zip(inputs, before))


def test_optional_gradients(moe):
    announce("linear: gradients one by one")
    c = Linear(moe, 200, 256, 320, 5)
    c.forward("gelu", True, False, True)
    c.backward("gelu")
    torch.cuda.synchronize()
    want = {n: c.o[n].clone() for n in ("dx", "dW", "db")}
    a, o = moe.MOET_ACT_GELU, c.o
    for n in want:
        c.o[n].fill_(77)
    moe.moet_linear_backward(c.p, None, c.W, o["u"], a, c.dy, o["dx"], None, None, o["wsb"])
    moe.moet_linear_backward(c.p, c.x, None, o["u"], a, c.dy, None, o["dW"], None, o["wsb"])
    moe.moet_linear_backward(c.p, None, None, o["u"], a, c.dy, None, None, o["db"], o["wsb"])
    torch.cuda.synchronize()
    for n, v in want.items():
        assert torch.equal(c.o[n], v), n
    # without activation u is not needed
    c.backward("none")
    torch.cuda.synchronize()
    want = {n: c.o[n].clone() for n in ("dx", "dW", "db")}
    moe.moet_linear_backward(c.p, c.x, c.W, None, moe.MOET_ACT_NONE, c.dy, o["dx"], o["dW"], o["db"], o["wsb"])
    torch.cuda.synchronize()
    for n, v in want.items():
        assert torch.equal(c.o[n], v), n


def test_slopes_of_far_arguments(moe):
    """Slopes where the sigmoid has saturated, at 0, and of infinities of u's range."""
    announce("linear: far arguments")
    vals = [0.0, -0.0, 1e-30, 5.0, -5.0, 30.0, -30.0, 1e4, -1e4, 3e38, -3e38, 0.7, -0.75, 1.4]
    c = Linear(moe, 16, 64, 64, 6)
    c.o["u"].copy_(torch.tensor((vals * 74)[:1024], device="cuda").view(16, 64))
    for act in ACTS:
        moe.moet_linear_backward(c.p, None, None, c.o["u"], code(moe, act), c.dy, None, None, c.o["db"], c.o["wsb"])
        torch.cuda.synchronize()
        with np.errstate(over="ignore", invalid="ignore"):
            slope = to.act_slope(np.clip(f64(c.o["u"]), -1e5, 1e5), act)
        db = (f64(c.dy) * slope).sum(0)
        e = (2.0 ** -17 + 60 * U32) * np.abs(f64(c.dy)).sum(0) * 1.13
        assert_within(act, f64(c.o["db"]), db, e + H * np.abs(db))


def test_gradients_against_differences(moe):
    """The loss sum(y c) of the operator's own outputs, in directions long enough for bfloat16 outputs to show."""
    announce("linear: differences")
    for act in ACTS:
        T, K, N = 64, 64, 128
        c = Linear(moe, T, K, N, 7)
        c.forward(act, True, False, True)
        c.backward(act)
        torch.cuda.synchronize()
        x, W, b, dy = f64(c.x), f64(c.W), f64(c.bias), f64(c.dy)
        g = np.random.default_rng(8)
        for name, v, grad in (("x", x, "dx"), ("W", W, "dW"), ("bias", b, "db")):
            d = g.normal(size=v.shape)
            h = 1e-6
            at = lambda s: np.sum(dy * to.act((x + s * d * (name == "x") if name == "x" else x) @  # noqa: E731
                                              (W + s * d if name == "W" else W) + (b + s * d if name == "bias" else b), act))
            num = (at(h) - at(-h)) / (2 * h)
            got = np.sum(f64(c.o[grad]) * d)
            # each gradient's value is off by at most about two half steps, independent of d's signs; u's rounding moves
            # a slope by half a step of u times 1.13, and relu's slope at the borders not at all here
            slack = 3 * H * np.sum(np.abs(f64(c.o[grad]) * d)) + 2 * H * np.sqrt(np.sum(d * d)) * np.sqrt(np.sum(dy * dy)) * 0.3
            assert abs(num - got) <= slack, (act, name, num, got)


def test_streams_and_graph_replays(moe):
    announce("linear on a side stream and captured")
    a, b = Linear(moe, 300, 320, 448, 9), Linear(moe, 4, 1024, 256, 10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.forward("gelu", True, True, True, s)
    a.backward("gelu", s)
    b.forward("gelu", True, True, True)
    b.backward("gelu")
    s.synchronize()
    for c in (a, b):
        c.check_forward("gelu", True, True, True)
        c.check_backward("gelu")
    names = ("u", "y", "dx", "dW", "db")
    want = [{n: c.o[n].clone() for n in names} for c in (a, b)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in (a, b):
            c.forward("gelu", True, True, True)
            c.backward("gelu")
    for _ in range(4):
        for c in (a, b):
            for n in c.o:
                c.o[n].view(torch.uint8).fill_(0x3F)
        g.replay()
        torch.cuda.synchronize()
        for c, w in zip((a, b), want):
            for n in names:
                assert torch.equal(c.o[n], w[n]), n


def test_the_same_bits_every_time(moe):
    announce("linear repeated")
    for T, K, N in ((1, 2048, 2048), (200, 2048, 512), (512, 2048, 1024)):
        c = Linear(moe, T, K, N, 11)
        got = []
        for _ in range(3):
            c.forward("gelu", True, True, True)
            c.backward("gelu")
            torch.cuda.synchronize()
            got.append([c.o[n].clone() for n in ("u", "y", "dx", "dW", "db")])
        assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(g, got[0]))
