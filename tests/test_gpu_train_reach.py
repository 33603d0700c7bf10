"""Calls that the documentation of moe_train.h allows and that lie at the edges of its
kernels: many selections a token, one step along K in many rounds of tiles, long
contractions, workspaces shared by captured graphs, norms past float32."""

import numpy as np
import pytest
import torch

from ext_helpers import assert_within, gen, randn
from gpu_helpers import U32, announce, f64, i64, needs_gpu
from oracle import train_ops as to
from test_gpu_adamw import LR, params_of
from test_gpu_linear import Linear
from test_gpu_tokens import Tokens

pytestmark = [pytest.mark.gpu, needs_gpu]

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T,d,E,k,drop,repeats", [(3, 64, 256, 256, 0.1, False), (50, 2048, 64, 20, 0.1, False),
                                                  (1030, 1088, 16, 16, 0.2, True), (2, 4096, 4, 4, 0.0, True)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_many_selections(moe, T, d, E, k, drop, repeats, dtype):
    announce(f"tokens T={T} d={d} E={E} k={k} repeats={repeats} {dtype}")
    t = Tokens(moe, T, d, E, k, dtype, 100, drop, repeats)
    t.run(True, True)
    t.check(True, True)


def test_every_selection_the_same_expert(moe):
    """One expert gets all rows, the deepest level of repeats, in more than one block of tokens."""
    announce("tokens: one expert for all")
    for T, k in ((9, 8), (600, 8)):
        t = Tokens(moe, T, 64, 8, k, F32, 101)
        t.idx.fill_(5)
        t.index = to.dispatch_index(i64(t.idx), 8)
        t.n = T * k
        t.rows.nan_to_num_(0.0)
        t.run(True, False)
        t.check(True, False)


def test_gates_of_one_expert(moe):
    """A softmax of one value: probability 1, gradient 0 but for what is added."""
    announce("gate backward E=1")
    p = moe.make_problem(100, 64, 1, 1, 64, F32)
    lg, dg, add = randn((100, 1), 3.0, F32, 1), randn((100, 1), 1.0, F32, 2), randn((100, 1), 1.0, F32, 3)
    out = torch.empty_like(lg)
    moe.moet_gate_backward(p, lg, torch.zeros(100, dtype=torch.int32, device="cuda"), dg, add, out)
    torch.cuda.synchronize()
    assert torch.equal(out, add)


@pytest.mark.parametrize("tile", ["0", "1", "2"])
@pytest.mark.parametrize("T,K,N", [(4352, 64, 4416), (4352, 4416, 64), (70, 4416, 4352)])
def test_rounds_of_short_tiles(moe, monkeypatch, tile, T, K, N):
    """One or two steps along K and several tiles a workgroup, in each of the three products."""
    announce(f"linear short tiles {tile} {T} {K} {N}")
    monkeypatch.setenv("MOE_LINEAR_TILE", tile)
    c = Linear(moe, T, K, N, 102)
    c.forward("gelu", True, True, True)
    c.check_forward("gelu", True, True, True)
    c.backward("gelu")
    c.check_backward("gelu")


def test_long_contraction_over_tokens(moe):
    announce("linear 100003 tokens")
    c = Linear(moe, 100003, 64, 64, 103)
    c.forward("silu", True, True, True)
    c.check_forward("silu", True, True, True)
    c.backward("silu")
    c.check_backward("silu")


def test_forced_tiles_that_cannot_be(moe, monkeypatch):
    """A forced tile whose launch the size does not fit falls back to the choice among all."""
    announce("linear forced tile out of reach")
    monkeypatch.setenv("MOE_LINEAR_TILE", "2")
    p = moe.make_problem(1 << 22, 64, 1, 1, 2048, BF)  # 2^23 tiles of 32 x 32: refused before (rows of 16 GiB)
    with pytest.raises(moe.MoEError):
        x = torch.empty(0, dtype=BF, device="cuda")
        moe.moet_linear(p, x.new_empty((1 << 22, 64)), x.new_empty((64, 2048)), None, 0, None, None, x.new_empty((1 << 22, 2048)),
                        torch.empty(moe.moet_workspace_size(p, moe.MOET_STAGE_LINEAR), dtype=torch.uint8, device="cuda"))
    p = moe.make_problem(1 << 18, 64, 1, 1, 2048, BF)  # 2^19 tiles: a launch of 2^28 threads
    x, W = randn((1 << 18, 64), 1.0, BF, 1), randn((64, 2048), 0.1, BF, 2)
    y = torch.empty((1 << 18, 2048), dtype=BF, device="cuda")
    ws = torch.empty(moe.moet_workspace_size(p, moe.MOET_STAGE_LINEAR), dtype=torch.uint8, device="cuda")
    moe.moet_linear(p, x, W, None, 0, None, None, y, ws)
    z = torch.empty_like(y)
    monkeypatch.delenv("MOE_LINEAR_TILE")
    moe.moet_linear(p, x, W, None, 0, None, None, z, torch.empty(
        moe.moet_workspace_size(p, moe.MOET_STAGE_LINEAR), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    # 64 products, one order of sums or another, and a rounding that may fall either side of a tie
    assert bool((y.float() - z.float()).abs().le(2.0 ** -7 * z.float().abs() + 64 * U32 * 64).all())


def test_graphs_that_share_a_workspace(moe):
    """Two captured calls with one workspace, replayed in turn, against their eager results."""
    announce("two graphs, one workspace")
    a, b = Linear(moe, 200, 2048, 512, 104), Linear(moe, 90, 2048, 512, 105)
    big = max((c.o[n] for c in (a, b) for n in ("ws", "wsb")), key=lambda t: t.numel())
    for c in (a, b):
        c.o["wsb"] = c.o["ws"] = big
        c.forward("gelu", True, True, True)
        c.backward("gelu")
    torch.cuda.synchronize()
    names = ("u", "y", "dx", "dW", "db")
    want = [{n: c.o[n].clone() for n in names} for c in (a, b)]
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.forward("gelu", True, True, True)
            c.backward("gelu")
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        c, w = (a, b)[i], want[i]
        for n in names:
            c.o[n].view(torch.uint8).fill_(0x5A)
        big.fill_(0xFF)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(c.o[n], w[n]) for n in names)


def test_norm_past_float32(moe):
    """Squares and a norm that float32 does not hold: the factor is still right, and the step is taken."""
    announce("grad norm of 3e39")
    g = torch.full((100,), 3e38, device="cuda")
    p = torch.zeros(100, device="cuda")
    opt = moe.AdamW([p], lr=LR, max_norm=1e30, weight_decay=0.0)
    norm = opt.step([g])
    torch.cuda.synchronize()
    assert torch.isinf(norm).item() and opt.counter.tolist() == [1, 0]
    want = 1e30 / float(np.sqrt(100.0) * np.float64(np.float32(3e38)))
    assert abs(float(opt.scale) - want) <= U32 * want
    # clipped to 1e29 each, whose squares float32 does not hold either: v is infinite, and m / sqrt(v) is 0
    assert torch.isinf(opt.v[0]).all() and not p.any()
    opt = moe.AdamW([p], lr=LR, max_norm=1.0, weight_decay=0.0)
    opt.step([g])
    torch.cuda.synchronize()
    assert bool((p + LR).abs().le(1e-4 * LR).all())  # 0.1 each: m / sqrt(v) is 1, eps 1e-7 of it


def test_two_optimizers_of_one_counter_are_refused_or_apart(moe):
    """A parameter twice in a list is refused; two lists with counters of their own run at once."""
    announce("adamw duplicates")
    params, grads = params_of([(5000, BF, BF), (300, F32, F32)], 15)
    opt = moe.AdamW([params[1], params[1]])
    with pytest.raises(moe.MoEError):
        opt.step([grads[1], grads[1]])
    wrong = moe.AdamW(params)
    state = wrong.state
    state["m"] = [state["m"][0][:100], state["m"][1]]
    with pytest.raises(ValueError, match="m holds"):
        moe.AdamW(params, state=state)
    with pytest.raises(ValueError, match="master"):
        moe.AdamW(params, state={**wrong.state, "master": [None, None]})
    with pytest.raises(moe.MoEError):  # not a multiple of 16 bytes
        moe.AdamW([params[1][1:]]).step([grads[1][1:]])


@pytest.mark.parametrize("T,E,K", [(77, 16, 4), (1, 8, 8)])
def test_block_of_odd_sizes(moe, T, E, K):
    from harness import make_inputs, scaled_config
    announce(f"train block T={T} E={E} k={K}")
    D, DE, DD = 320, 192, 448
    cfg = scaled_config("fine_grained", T=T, d_model=D, E=E, k=K, d_expert=DE, suffix="odd")
    inp = make_inputs(cfg, seed=2, device="cuda")
    P = {"gain": torch.ones(D, device="cuda").to(BF), **{n: inp[n] for n in ("w_router", "W1", "W2")},
         "V1": randn((D, DD), D ** -0.5, BF, 1), "c1": randn((DD,), 0.1, BF, 2), "V2": randn((DD, D), DD ** -0.5, BF, 3),
         "c2": randn((D,), 0.1, BF, 4)}
    block = moe.MoETrainBlock(T, D, E, K, DE, P, max_norm=1.0, bits=8)
    x, dy = randn((T, D), 1.0, BF, 5), randn((T, D), 1.0, BF, 6)
    y, _ = block.forward(x)
    dx = block.backward(dy)
    block.step()
    torch.cuda.synchronize()
    for t in (y, dx, *P.values(), *block.grads.values()):
        assert torch.isfinite(t.float()).all()
    n = block.n.float()
    # the dense expert's part of the output: what is not the routed experts'
    dense = (y.float() - block.routed.float())
    a = block.a.float()
    assert float((dense.norm())) > 0 and a.shape == (T, DD)
    # gradient of the second bias is the sum of dy, of bfloat16 values in float32 and rounded once
    s = f64(dy).sum(0)
    assert_within("c2", f64(block.grads["c2"]), s, (T + 40) * U32 * np.abs(f64(dy)).sum(0) + 2.0 ** -8 * np.abs(s))


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("pt,gt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_long_lists_take_the_same_step(moe, bits, pt, gt):
    """Lists of 8 million values and more (loads and stores past the caches): the bits of a short list's step, whose
    tensor is the beginning of theirs."""
    announce(f"adamw long list bits={bits} {pt} {gt}")
    n, m = (8 << 20) + 1237, 1 << 20
    g = gen(16)
    p = (torch.randn(n, generator=g, device="cuda") * 0.1).to(pt)
    gr = torch.randn(n, generator=g, device="cuda").to(gt)
    q, gq = p[:m].clone(), gr[:m].clone()
    a, b = (moe.AdamW([t], lr=LR, bits=[bits], seed=4) for t in (p, q))
    for _ in range(2):
        a.step([gr])
        b.step([gq])
    torch.cuda.synchronize()
    assert torch.equal(p[:m], q) and torch.equal(a.counter, b.counter)
    for x, y in ((a.m[0][:m], b.m[0]), (a.v[0][:m], b.v[0])):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.isfinite(p.float()).all() and bool((a.v[0][-2000:].float() > 0).all())
    # the tail, past the last whole chunk: as a tensor of its own, whose moments in 32 bits do not depend on its place
    if bits == 32:
        t = (n // 2048) * 2048
        c = moe.AdamW([torch.zeros(n - t, device="cuda")], lr=LR, bits=[32])
        for _ in range(2):
            c.step([gr[t:].clone()])
        torch.cuda.synchronize()
        assert torch.equal(a.m[0][t:], c.m[0]) and torch.equal(a.v[0][t:], c.v[0])
