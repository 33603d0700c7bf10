"""Rows sorted by expert and back on the GPU, with weights and gradients, against float64.

Bounds: a product or sum of n float32 terms is off by at most n 2^-24 of the sum of
magnitudes (2^-24 for each operation), and a result rounded to its type by half a step
of itself. A dot product over d values is added in chains of at most d / 64 + 8 values a
lane, six pairs of lanes and four waves.
"""

import numpy as np
import pytest
import torch

from ext_helpers import HALF, TINY, assert_within, gen, randn
from gpu_helpers import U32, announce, f64, i64, needs_gpu
from oracle import train_ops as to
from test_gpu_canary import Guarded

pytestmark = [pytest.mark.gpu, needs_gpu]

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def new(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


class Tokens:
    """Buffers and inputs of one shape; guarded: every output between bands of a known pattern."""

    def __init__(self, moe, T, d, E, k, dtype, seed, drop=0.0, repeats=False, guarded=False):
        self.moe, self.p = moe, moe.make_problem(T, d, E, k, 64, dtype)
        self.T, self.d, self.E, self.k, self.dtype = T, d, E, k, dtype
        g = gen(seed)
        if repeats:
            idx = torch.randint(0, E, (T, k), generator=g, device="cuda")
        else:
            idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k]
        gone = torch.rand((T, k), generator=g, device="cuda") < drop
        wrong = torch.where(torch.rand((T, k), generator=g, device="cuda") < 0.5, -1, E)
        self.idx = torch.where(gone, wrong, idx).to(I32).contiguous()
        self.gate = torch.rand((T, k), generator=g, device="cuda") * 2 - 0.5
        self.x, self.add, self.dy = (randn((T, d), 1.0, dtype, seed + i) for i in (1, 2, 3))
        self.rows = randn((T * k, d), 1.0, dtype, seed + 4)
        self.logits = randn((T, E), 2.0, F32, seed + 5)
        make = (lambda s, t: Guarded(s, t)) if guarded else (lambda s, t: new(s, t))
        self.out = {"counts": make((E,), I32), "offsets": make((E + 1,), I32), "perm": make((T * k,), I32),
                    "inv": make((T * k,), I32), "x_perm": make((T * k, d), dtype), "y": make((T, d), dtype),
                    "dy_perm": make((T * k, d), dtype), "dx": make((T, d), dtype), "dgate": make((T, k), F32),
                    "dweight": make((T, k), F32), "dlogits": make((T, E), F32),
                    "ws": make((moe.moet_workspace_size(self.p, moe.MOET_STAGE_DISPATCH),), torch.uint8)}
        self.o = {n: v.t if guarded else v for n, v in self.out.items()}
        for n in ("perm", "x_perm", "dy_perm"):
            self.o[n].zero_()
        i = to.dispatch_index(i64(self.idx), E)
        self.index, self.n = i, i["perm"].size
        # rows that no selection names: never read
        self.rows[self.n:] = float("nan")

    def run(self, weighted, residual, stream=None):
        m, p, o = self.moe, self.p, self.o
        w = self.gate if weighted else None
        add = self.add if residual else None
        m.moet_dispatch(p, self.idx, w, self.x, o["counts"], o["offsets"], o["perm"], o["inv"], o["x_perm"], o["ws"], stream)
        m.moet_combine(p, self.rows, o["inv"], w, add, o["y"], stream)
        m.moet_combine_backward(p, self.dy, o["inv"], self.rows, w, o["dy_perm"], o["dgate"], stream)
        m.moet_dispatch_backward(p, self.rows, o["inv"], self.x, w, add, o["dx"], o["dweight"], stream)
        m.moet_gate_backward(p, self.logits, self.idx, o["dgate"], self.logits if residual else None, o["dlogits"], stream)
        return o

    def check(self, weighted, residual):
        torch.cuda.synchronize()
        o, i, n, T, k, d, E = self.o, self.index, self.n, self.T, self.k, self.d, self.E
        half = HALF[self.dtype]
        for name in ("counts", "offsets", "inv"):
            assert np.array_equal(i64(o[name]), i[name]), name
        perm = i64(o["perm"])
        assert np.array_equal(perm[:n], i["perm"]) and not perm[n:].any()
        w = f64(self.gate) if weighted else None
        aw = np.abs(w) if weighted else None
        for name, src in (("x_perm", self.x), ("dy_perm", self.dy)):
            ref = to.to_rows(f64(src), i, w)
            got = f64(o[name])
            err = (half + U32) * np.abs(ref) + TINY if weighted else 0.0
            assert_within(name, got[:n], ref, err)
            assert not got[n:].any(), name  # untouched
        rows = f64(self.rows)
        add = f64(self.add) if residual else None
        ref = to.from_rows(rows, i, w, add, T)
        mag = to.from_rows(np.abs(rows), i, aw, None if add is None else np.abs(add), T)
        bound = (k + 2) * U32 * mag + half * (np.abs(ref) + (k + 2) * U32 * mag)
        assert_within("y", f64(o["y"]), ref, bound)
        assert_within("dx", f64(o["dx"]), ref, bound)
        for name, tok in (("dgate", self.dy), ("dweight", self.x)):
            ref = to.dots(rows, f64(tok), i, k)
            mag = to.dots(np.abs(rows), np.abs(f64(tok)), i, k)
            assert_within(name, f64(o[name]), ref, (d / 64 + 8 + 12) * U32 * mag + U32 * np.abs(ref))
        # softmax: differences of logits, exponential and reciprocal within 2^-22 and the rounding of the difference,
        # sums of E terms; then p (dp - mean) from two such sums
        lg, dg = f64(self.logits), f64(o["dgate"])
        ref = to.gate_backward(lg, i64(self.idx), dg, lg if residual else None)
        q = to.softmax_rows(lg)
        dp = np.abs(to.gate_backward(lg * 0, i64(self.idx), dg, None))  # shape only
        mags = np.zeros((T, E))
        for j in range(k):
            e = i64(self.idx)[:, j]
            ok = (e >= 0) & (e < E)
            np.add.at(mags, (np.nonzero(ok)[0], e[ok]), np.abs(dg[ok, j]))
        spread = np.max(lg, 1, keepdims=True) - lg
        rel = (64 + E / 64 + k + 2 * spread.max()) * U32
        bound = rel * q * (mags + np.sum(q * mags, 1, keepdims=True)) + 2 * U32 * (np.abs(ref) + (np.abs(lg) if residual else 0)) + TINY
        assert_within("dlogits", f64(o["dlogits"]), ref, bound)
        assert dp.shape == mags.shape


# T, d, E, k, dropped, repeated experts
SHAPES = [
    (1, 64, 1, 1, 0.0, False), (1, 7168, 8, 8, 0.0, False), (3, 128, 5, 5, 0.5, False), (7, 64, 16, 12, 0.2, False),
    (32, 2048, 64, 8, 0.0, False), (33, 576, 200, 3, 0.1, False), (300, 320, 12, 3, 1.0, False),
    (777, 320, 12, 3, 0.1, False), (1025, 64, 8, 2, 0.3, False), (2100, 192, 256, 8, 0.1, False),
    (40, 128, 6, 6, 0.2, True), (1500, 64, 8, 8, 0.1, True), (700, 64, 40, 40, 0.0, True), (17000, 64, 8, 2, 0.0, False),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,drop,repeats", SHAPES)
def test_against_float64(moe, T, d, E, k, drop, repeats, dtype):
    announce(f"tokens T={T} d={d} E={E} k={k} drop={drop} repeats={repeats} {dtype}")
    t = Tokens(moe, T, d, E, k, dtype, 10, drop, repeats)
    for weighted, residual in ((True, True), (False, False)):
        for n in ("perm", "x_perm", "dy_perm"):
            t.o[n].zero_()
        t.run(weighted, residual)
        t.check(weighted, residual)


@pytest.mark.parametrize("T,k", [(5, 2), (900, 4)])
def test_only_outputs_are_written(moe, T, k):
    announce(f"tokens guarded T={T} k={k}")
    t = Tokens(moe, T, 320, 12, k, BF, 20, 0.2, guarded=True)
    inputs = {n: getattr(t, n) for n in ("idx", "gate", "x", "add", "dy", "rows", "logits")}
    before = {n: v.clone() for n, v in inputs.items()}
    t.run(True, True)
    t.check(True, True)
    for n, g in t.out.items():
        assert g.intact(), n
    for n, v in inputs.items():
        assert torch.equal(v.view(torch.uint8), before[n].view(torch.uint8)), n


def test_optional_outputs(moe):
    """Gradients of the rows alone, as a caller without gates' gradients asks for them."""
    announce("tokens without dgate")
    t = Tokens(moe, 300, 128, 8, 2, BF, 30)
    o = {n: v.clone() for n, v in t.run(True, False).items()}
    dp, dx = torch.zeros_like(o["dy_perm"]), torch.empty_like(o["dx"])
    moe.moet_combine_backward(t.p, t.dy, o["inv"], None, t.gate, dp, None)
    moe.moet_dispatch_backward(t.p, t.rows, o["inv"], None, t.gate, None, dx, None)
    torch.cuda.synchronize()
    assert torch.equal(dp, o["dy_perm"]) and torch.equal(dx, o["dx"])


def test_index_is_the_layers(moe):
    """Distinct experts: the same index and rows as moe_permute, bit for bit."""
    announce("tokens against moe_permute")
    for T, k in ((20, 2), (3000, 4)):
        t = Tokens(moe, T, 128, 16, k, BF, 40)
        t.run(False, False)
        o = [new(s, I32) for s in ((16,), (17,), (T * k,), (T * k,))] + [new((T * k, 128), BF)]
        ws = new((moe.moe_workspace_size(t.p, moe.MOE_STAGE_PERMUTE),), torch.uint8)
        moe.moe_permute(t.p, t.idx, t.x, *o, ws)
        torch.cuda.synchronize()
        for name, v in zip(("counts", "offsets", "perm", "inv", "x_perm"), o):
            assert torch.equal(v, t.o[name]), name


def test_rows_out_of_range_are_dropped(moe):
    """Entries of inv outside [0, T k) name no row, in every call."""
    announce("tokens inv out of range")
    t = Tokens(moe, 64, 128, 8, 2, F32, 50)
    inv = torch.full((128,), -1, dtype=I32, device="cuda")
    inv[::3] = 128
    inv[1::3] = 2 ** 31 - 1
    inv[2::3] = -2 ** 31
    y, dx, dg = new((64, 128), F32), new((64, 128), F32), new((64, 2), F32)
    rows = torch.full((128, 128), 7.0, device="cuda")
    moe.moet_combine(t.p, t.rows, inv, t.gate, t.add, y)
    moe.moet_combine_backward(t.p, t.dy, inv, t.rows, t.gate, rows, dg)
    torch.cuda.synchronize()
    assert torch.equal(y, t.add) and bool((rows == 7).all()) and not dg.any()
    moe.moet_dispatch_backward(t.p, t.rows, inv, t.x, None, None, dx, dg)
    torch.cuda.synchronize()
    assert not dx.any() and not dg.any()


def test_infinities_and_empty_rows_of_logits(moe):
    announce("gate backward with -inf")
    T, E, k = 70, 40, 3
    p = moe.make_problem(T, 64, E, k, 64, F32)
    lg = randn((T, E), 2.0, F32, 60)
    lg[:, 5:9] = float("-inf")
    lg[7] = float("-inf")
    idx = torch.rand((T, E), generator=gen(61), device="cuda").argsort(1)[:, :k].to(I32).contiguous()
    idx[3] = -1
    dg = randn((T, k), 1.0, F32, 62)
    dg[3] = float("nan")  # of dropped selections: not read
    out = new((T, E), F32)
    moe.moet_gate_backward(p, lg, idx, dg, None, out)
    torch.cuda.synchronize()
    ref = to.gate_backward(f64(lg), i64(idx), f64(dg), None)
    got = f64(out)
    assert not got[7].any() and not got[3].any() and not got[:, 5:9].any()
    assert_within("dlogits", got, ref, 200 * U32 * np.abs(f64(dg)[~np.isnan(f64(dg))]).sum() / T + TINY)


def test_gradients_against_differences(moe):
    """d(sum of y c) / d(x, gate, y_perm) by central differences of the float32 calls themselves."""
    announce("tokens differences")
    T, d, E, k = 6, 64, 4, 2
    t = Tokens(moe, T, d, E, k, F32, 70, 0.2)
    t.rows.nan_to_num_(0.0)
    o = t.run(True, False)
    torch.cuda.synchronize()
    inv, dg, dyp = o["inv"].clone(), o["dgate"].clone(), o["dy_perm"].clone()

    def loss(rows, gate):
        y = new((T, d), F32)
        moe.moet_combine(t.p, rows, inv, gate, None, y)
        return float((y.double() * t.dy.double()).sum())

    h = 2.0 ** -4  # linear in each: only rounding, 2^-24 of sums of about 100 terms over 2 h
    for a in range(T):
        for j in range(k):
            up, dn = t.gate.clone(), t.gate.clone()
            up[a, j] += h
            dn[a, j] -= h
            assert abs((loss(t.rows, up) - loss(t.rows, dn)) / (2 * h) - float(dg[a, j])) < 1e-3
    for r in range(0, t.n, 3):
        for c in (0, 17, 63):
            up, dn = t.rows.clone(), t.rows.clone()
            up[r, c] += h
            dn[r, c] -= h
            assert abs((loss(up, t.gate) - loss(dn, t.gate)) / (2 * h) - float(dyp[r, c])) < 1e-3


def test_streams_and_graph_replays(moe):
    announce("tokens on a side stream and captured")
    a, b = Tokens(moe, 900, 256, 16, 4, BF, 80, 0.1), Tokens(moe, 20, 256, 16, 4, BF, 81, 0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.run(True, True, s)   # two calls at once
    b.run(True, True)
    s.synchronize()
    a.check(True, True)
    b.check(True, True)
    want = [{n: v.clone() for n, v in t.o.items() if n != "ws"} for t in (a, b)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(True, True)
        b.run(True, True)
    for _ in range(4):
        for t in (a, b):
            for n, v in t.o.items():
                if n not in ("perm", "x_perm", "dy_perm"):
                    v.view(torch.uint8).fill_(0x5A)
        g.replay()
        torch.cuda.synchronize()
        for t, w in zip((a, b), want):
            for n, v in w.items():
                assert torch.equal(t.o[n], v), n
    torch.randn(1000, device="cuda").sum().item()


def test_rows_past_32_bit_offsets(moe):
    """T k rows of 2^32 values and more (the last rows' values against the tokens')."""
    T, k, d = 40000, 8, 14336
    announce("tokens past 2^32 values")
    p = moe.make_problem(T, d, 8, k, 64, BF)
    idx = torch.arange(k, device="cuda", dtype=I32).repeat(T, 1).contiguous()
    x = randn((T, d), 1.0, BF, 90)
    o = [new(s, I32) for s in ((8,), (9,), (T * k,), (T * k,))]
    rows = new((T * k, d), BF)
    ws = new((moe.moet_workspace_size(p, moe.MOET_STAGE_DISPATCH),), torch.uint8)
    moe.moet_dispatch(p, idx, None, x, *o, rows, ws)
    assert rows.numel() >= 1 << 32
    assert torch.equal(rows[7 * T:], x) and torch.equal(rows[5 * T:6 * T], x)
    y, dg = new((T, d), BF), new((T, k), F32)
    moe.moet_combine(p, rows, o[3], torch.full((T, k), 0.125, device="cuda"), None, y)
    assert torch.equal(y, x)
    moe.moet_dispatch_backward(p, rows, o[3], x, None, None, y, dg)
    assert torch.equal(y, 8 * x)  # exact: eight equal values
    sq = x.float().square().sum(1)
    assert bool((dg - sq[:, None]).abs().le((d / 64 + 20) * U32 * sq[:, None]).all())


def test_stages_make_the_layer(moe):
    """moe_route, dispatch, experts of the caller's own, combine and the gradients back, against the layer's backward."""
    from harness import make_dense, make_inputs, scaled_config
    announce("stages against moe_backward")
    T, d, E, k, de = 200, 256, 8, 2, 128
    cfg = scaled_config("fine_grained", T=T, d_model=d, E=E, k=k, d_expert=de, suffix="stages")
    inp = make_inputs(cfg, seed=5, device="cuda")
    dy = make_dense((T, d), 1.0, seed=5, tag=3, device="cuda")
    p = moe.make_problem(T, d, E, k, de, BF)
    y, dx = new((T, d), BF), new((T, d), BF)
    dwr, dW1, dW2 = (torch.empty_like(inp[n]) for n in ("w_router", "W1", "W2"))
    dbias, logits = new((E,), F32), new((T, E), F32)
    ws = new((moe.moe_workspace_size(p, moe.MOE_STAGE_TRAIN),), torch.uint8)
    moe.moe_forward_train(p, inp["x"], inp["w_router"], None, inp["W1"], inp["W2"], y, ws)
    moe.moe_backward(p, inp["x"], inp["w_router"], inp["W1"], inp["W2"], dy, dx, dwr, dbias, dW1, dW2, None, None, ws)
    idx, gate = new((T, k), I32), new((T, k), F32)
    ws_r = new((moe.moe_workspace_size(p, moe.MOE_STAGE_ROUTE),), torch.uint8)
    moe.moe_route_ws(p, inp["x"], inp["w_router"], None, logits, idx, gate, ws_r)
    o = [new(s, I32) for s in ((E,), (E + 1,), (T * k,), (T * k,))]
    x_perm = new((T * k, d), BF)
    ws_d = new((moe.moet_workspace_size(p, moe.MOET_STAGE_DISPATCH),), torch.uint8)
    moe.moet_dispatch(p, idx, None, inp["x"], *o, x_perm, ws_d)
    lim = o[1].tolist()
    leaf = x_perm.float().requires_grad_()
    W1, W2 = (inp[n].float().requires_grad_() for n in ("W1", "W2"))
    outs = [torch.nn.functional.gelu(leaf[lim[e]:lim[e + 1]] @ W1[e], approximate="tanh") @ W2[e] for e in range(E)]
    y_perm = torch.cat(outs)
    rows = y_perm.detach().to(BF)
    y2, dyp, dgate, dlog, dx2 = new((T, d), BF), new((T * k, d), BF), new((T, k), F32), new((T, E), F32), new((T, d), BF)
    moe.moet_combine(p, rows, o[3], gate, None, y2)
    moe.moet_combine_backward(p, dy, o[3], rows, gate, dyp, dgate)
    moe.moet_gate_backward(p, logits, idx, dgate, None, dlog)
    y_perm.backward(dyp.float())
    through_router = (dlog @ inp["w_router"].float().t().contiguous()).to(BF)
    moe.moet_dispatch_backward(p, leaf.grad.to(BF), o[3], None, None, through_router, dx2, None)
    torch.cuda.synchronize()
    # the two ways round their intermediates to bf16 at different places: a few half steps in the norm
    for name, a, b in (("y", y2, y), ("dx", dx2, dx), ("dW1", W1.grad, dW1), ("dW2", W2.grad, dW2),
                       ("dbias", dlog.sum(0), dbias), ("dw_router", inp["x"].float().t().contiguous() @ dlog, dwr)):
        err = float((a.float() - b.float()).norm() / b.float().norm())
        assert err < 6 * HALF[BF], (name, err)
