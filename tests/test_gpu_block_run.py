"""The operators used together as a block: norm with residual -> layer with 8-bit
experts -> next norm; a training step with the balance loss; graph replay, other
streams, two calls at once; and that nothing but outputs is written."""

import numpy as np
import pytest
import torch

import oracle
from ext_helpers import HALF, assert_within, f64, ffn_bound, randn
from gpu_helpers import U32, announce, logit_bound, needs_gpu, rel_err
from harness import host_array, make_dense, make_inputs, scaled_config
from oracle import block_ops as ob
from test_gpu_canary import Guarded, check

pytestmark = [pytest.mark.gpu, needs_gpu]

BF, F32 = torch.bfloat16, torch.float32


class Block:
    """Buffers of norm + 8-bit layer for one shape."""

    def __init__(self, moe, T, d, E, k, de, seed):
        self.moe, self.p = moe, moe.make_problem(T, d, E, k, de, BF)
        cfg = scaled_config("fine_grained", T=T, d_model=d, E=E, k=k, d_expert=de, suffix="block")
        inp = make_inputs(cfg, seed=seed, device="cuda")
        self.cfg, self.wr, self.W1, self.W2 = cfg, inp["w_router"], inp["W1"], inp["W2"]
        self.gain = (1 + 0.1 * randn((d,), 1.0, F32, seed + 1)).to(BF)
        self.q = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in moe.expert_shapes(self.p)]
        moe.moex_quantize_experts(self.p, self.W1, self.W2, *self.q)
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
        self.h, self.n, self.y = new((T, d), BF), new((T, d), BF), new((T, d), BF)
        self.n8, self.ns = new((T, moe.code_pitch(d)), torch.uint8), new((T, moe.scale_pitch(d)), torch.uint8)
        self.ws = new((moe.moex_workspace_size(self.p, moe.MOEX_STAGE_FORWARD_FP8),), torch.uint8)

    def __call__(self, x, res, stream=None):
        m = self.moe
        m.moex_add_rmsnorm(self.p, x, res, self.gain, 1e-6, self.h, self.n, self.n8, self.ns, None, stream)
        m.moex_forward_fp8(self.p, self.n, self.n8, self.ns, self.wr, None, *self.q, self.y, self.ws, stream)
        return self.y


SHAPES = [(1, 256, 16, 4, 128), (7, 320, 8, 2, 448), (300, 512, 16, 4, 320), (1500, 256, 8, 2, 256)]


@pytest.mark.parametrize("T,d,E,k,de", SHAPES)
def test_block_against_float64(moe, T, d, E, k, de):
    announce(f"block T={T} d={d} E={E} k={k} de={de}")
    b = Block(moe, T, d, E, k, de, 1)
    x, res = randn((T, d), 1.0, BF, 5), randn((T, d), 1.0, BF, 6)
    y = b(x, res).clone()
    # the same without the norm's 8-bit rows: made by the layer call from the bf16 rows
    y_own = torch.empty_like(y)
    moe.moex_forward_fp8(b.p, b.n, None, None, b.wr, None, *b.q, y_own, b.ws)
    torch.cuda.synchronize()
    n = f64(b.n)
    route = oracle.route(f64(b.n), f64(b.wr), None, k)
    idx, gate, tie = route["idx"], route["gate"], route["near_tie"]
    pm = oracle.permute(idx.astype(np.int64), E)
    w1, w2 = ob.weight_layout(f64(b.W1))[2], ob.weight_layout(f64(b.W2))[2]
    sb = b.ns.cpu().numpy().astype(np.int64)[:, :moe.code_pitch(d) // 128] - 127
    for rows, got in ((ob.decode(b.n8.cpu().numpy(), sb), y), (ob.decode(*ob.encode(n)), y_own)):
        # the expert rows' own bound (a hidden value near the border of two codes may take either, a step of
        # 2^-3 of it), carried through the combine: gates off by twice the logits' rounding and the softmax's
        # units, k float32 products and additions, one rounding to bf16
        yp, bound = ffn_bound(rows[pm["perm"]], pm["offsets"], w1, w2, de)
        ref, mag = oracle.combine(yp, pm["inv"], gate), oracle.combine(np.abs(yp), pm["inv"], gate)
        dg = 2 * logit_bound(n, f64(b.wr), None, route["logits"]).max(axis=1, keepdims=True) + 32 * U32
        assert_within("y", f64(got)[~tie], ref[~tie],
                      (oracle.combine(bound, pm["inv"], gate) * (1 + dg) + (dg + 2 * k * U32) * mag
                       + HALF[BF] * (np.abs(ref) + 2.0 ** -6 * mag))[~tie])
    # and the 8-bit experts stay near the bf16 layer: three roundings of 2^-4 at most each, mostly cancelling
    full = oracle.forward(host_array(b.n), host_array(b.wr), None, host_array(b.W1), host_array(b.W2), k, "bf16")
    err = np.linalg.norm(f64(y)[~tie] - full["y"][~tie]) / np.linalg.norm(full["y"][~tie])
    assert err <= 0.0625 * 3


def test_two_blocks_chain(moe):
    """The second block's norm adds the first block's output to its stream."""
    announce("block chain")
    T, d = 50, 256
    a, c = Block(moe, T, d, 8, 2, 128, 3), Block(moe, T, d, 8, 2, 128, 4)
    x, res = randn((T, d), 1.0, BF, 7), randn((T, d), 1.0, BF, 8)
    a(x, res)
    c(a.y, a.h)
    torch.cuda.synchronize()
    assert torch.equal(c.h, (a.y.float() + a.h.float()).to(BF))
    y, r = ob.rmsnorm(f64(c.h), f64(c.gain), 1e-6)
    assert rel_err(f64(c.n), y) <= 2.0 ** -8
    assert torch.isfinite(c.y).all()


def test_block_class_is_the_two_calls(moe):
    announce("MoEBlockFP8")
    T, d, E, k, de = 70, 320, 8, 2, 448
    b = Block(moe, T, d, E, k, de, 2)
    m = moe.MoEBlockFP8(T, d, E, k, de, b.gain, b.wr, b.W1, b.W2)
    x, res = randn((T, d), 1.0, BF, 9), randn((T, d), 1.0, BF, 10)
    b(x, res)
    y, h = m(x, res)
    torch.cuda.synchronize()
    assert torch.equal(y, b.y) and torch.equal(h, b.h)
    y2, h2 = m(b.h)  # without a residual the stream is x itself: the same rows, the same result
    torch.cuda.synchronize()
    assert h2 is b.h and torch.equal(y2, b.y)


@pytest.mark.parametrize("T,d,E,k,de", [(4, 256, 16, 4, 128), (600, 512, 16, 4, 320)])
def test_graph_replay(moe, T, d, E, k, de):
    announce(f"block graph T={T}")
    b, e = Block(moe, T, d, E, k, de, 5), Block(moe, T, d, E, k, de, 5)
    xs = [(randn((T, d), 1.0, BF, 20 + i), randn((T, d), 1.0, BF, 40 + i)) for i in range(3)]
    x, res = xs[0][0].clone(), xs[0][1].clone()
    logits, idx = randn((T, E), 1.0, F32, 60), torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
    p = moe.make_problem(T, d, E, k, de, BF)
    bw = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_BALANCE), dtype=torch.uint8, device="cuda")
    nw = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_NORM_BACKWARD), dtype=torch.uint8, device="cuda")

    def rest(o):
        moe.moex_balance_loss(p, logits, idx, None, 0.1, o["loss"], o["counts"], o["mp"], o["dl"], bw)
        moe.moex_add_rmsnorm_backward(p, x, b.gain, o["r"], res, None, o["dx"], o["dg"], nw)

    def outs():
        return {"loss": torch.zeros(1, device="cuda"), "counts": torch.zeros(E, dtype=torch.int32, device="cuda"),
                "mp": torch.zeros(E, device="cuda"), "dl": torch.zeros((T, E), device="cuda"),
                "r": torch.ones(T, device="cuda"), "dx": torch.zeros_like(x), "dg": torch.zeros(d, device="cuda")}

    og, oe = outs(), outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            b(x, res)
            rest(og)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b(x, res)
        rest(og)
    torch.cuda.synchronize()
    for i in [1, 2, 0, 1]:
        x.copy_(xs[i][0])
        res.copy_(xs[i][1])
        logits.add_(0.25)
        logits[:, 0].mul_(1.5)
        junk = torch.randn(4096, device="cuda").sum()
        graph.replay()
        torch.cuda.synchronize()
        e(xs[i][0], xs[i][1])
        rest(oe)
        torch.cuda.synchronize()
        assert torch.equal(b.y, e.y) and torch.equal(b.h, e.h), i
        for key in og:
            assert torch.equal(og[key], oe[key]), (i, key)
        assert torch.isfinite(junk)


def test_two_streams_at_once(moe):
    """Two blocks with buffers of their own on two streams, interleaved."""
    announce("block two streams")
    T, d = 200, 256
    blocks = [Block(moe, T, d, 8, 2, 256, 6) for _ in range(2)]
    xs = [(randn((T, d), 1.0, BF, 70 + i), randn((T, d), 1.0, BF, 80 + i)) for i in range(2)]
    alone = []
    for b, (x, r) in zip(blocks, xs):
        alone.append(b(x, r).clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(5):
        for b, (x, r), s in zip(blocks, xs, streams):
            b(x, r, s)
    torch.cuda.synchronize()
    for b, want in zip(blocks, alone):
        assert torch.equal(b.y, want)


@pytest.mark.parametrize("T,d,E,k,de", [(5, 192, 12, 3, 320), (333, 320, 16, 4, 448)])
def test_only_outputs_are_written(moe, T, d, E, k, de):
    announce(f"canary ext T={T} d={d} E={E} k={k} de={de}")
    p = moe.make_problem(T, d, E, k, de, BF)
    cfg = scaled_config("skewed", T=T, d_model=d, E=E, k=k, d_expert=de, suffix="ext")
    inp = make_inputs(cfg, seed=23, device="cuda")
    x, wr, bias, W1, W2 = inp["x"], inp["w_router"], inp["router_bias"], inp["W1"], inp["W2"]
    res, gain, dy = randn((T, d), 1.0, BF, 1), randn((d,), 1.0, BF, 2), randn((T, d), 1.0, BF, 3)
    u8, i32 = torch.uint8, torch.int32
    wsg = lambda stage: Guarded((moe.moex_workspace_size(p, stage),), u8)  # noqa: E731

    def run(name, g, ins, f):
        before = {n: t.clone() for n, t in ins.items()}
        f({n: v.t for n, v in g.items()})
        check(name, g, ins, before)
        return {n: v.t.clone() for n, v in g.items()}

    cp, sp = moe.code_pitch(d), moe.scale_pitch(d)
    for dt, xx, rr, gg, dd in ((BF, x, res, gain, dy), (F32, x.float(), res.float(), gain.float(), dy.float())):
        pn = moe.make_problem(T, d, E, k, de, dt)
        o = run("norm", {"h": Guarded((T, d), dt), "y": Guarded((T, d), dt), "y8": Guarded((T, cp), u8),
                         "ys": Guarded((T, sp), u8), "r": Guarded((T,), F32)}, {"x": xx, "res": rr, "gain": gg},
                lambda t: moe.moex_add_rmsnorm(pn, xx, rr, gg, 1e-6, t["h"], t["y"], t["y8"], t["ys"], t["r"]))
        run("norm backward", {"dx": Guarded((T, d), dt), "dg": Guarded((d,), F32),
                              "ws": wsg(moe.MOEX_STAGE_NORM_BACKWARD)},
            {"h": o["h"], "gain": gg, "r": o["r"], "dy": dd, "dh": rr},
            lambda t: moe.moex_add_rmsnorm_backward(pn, o["h"], gg, o["r"], dd, rr, t["dx"], t["dg"], t["ws"]))
        q = run("quantize rows", {"x8": Guarded((T, cp), u8), "xs": Guarded((T, sp), u8)}, {"x": xx},
                lambda t: moe.moex_quantize_rows(pn, xx, t["x8"], t["xs"]))
    logits, idx = randn((T, E), 1.0, F32, 5), torch.randint(0, E, (T, k), device="cuda", dtype=i32)
    mask = (torch.rand(T, device="cuda") < 0.8).to(u8)
    run("balance", {"loss": Guarded((1,), F32), "c": Guarded((E,), i32), "mp": Guarded((E,), F32),
                    "dl": Guarded((T, E), F32), "ws": wsg(moe.MOEX_STAGE_BALANCE)},
        {"logits": logits, "idx": idx, "mask": mask},
        lambda t: moe.moex_balance_loss(p, logits, idx, mask, 0.1, t["loss"], t["c"], t["mp"], t["dl"], t["ws"]))
    s1, c1, s2, c2 = moe.expert_shapes(p)
    w = run("quantize experts", {"W1q": Guarded(s1, u8), "W1s": Guarded(c1, u8), "W2q": Guarded(s2, u8),
                                 "W2s": Guarded(c2, u8)}, {"W1": W1, "W2": W2},
            lambda t: moe.moex_quantize_experts(p, W1, W2, t["W1q"], t["W1s"], t["W2q"], t["W2s"]))
    R = T * k
    perm = torch.randint(0, T, (R,), device="cuda", dtype=i32)
    off = torch.linspace(0, R, E + 1, device="cuda").to(i32)
    run("ffn", {"y": Guarded((R, d), BF), "ws": wsg(moe.MOEX_STAGE_FFN_FP8)},
        dict(w, x8=q["x8"], xs=q["xs"], perm=perm, off=off),
        lambda t: moe.moex_grouped_ffn_fp8(p, q["x8"], q["xs"], perm, off, w["W1q"], w["W1s"], w["W2q"], w["W2s"],
                                           t["y"], t["ws"]))
    ins = dict(w, x=x, x8=q["x8"], xs=q["xs"], wr=wr)
    if bias is not None:
        ins["bias"] = bias
    run("forward", {"y": Guarded((T, d), BF), "ws": wsg(moe.MOEX_STAGE_FORWARD_FP8)}, ins,
        lambda t: moe.moex_forward_fp8(p, x, q["x8"], q["xs"], wr, bias, w["W1q"], w["W1s"], w["W2q"], w["W2s"],
                                       t["y"], t["ws"]))
    if E % 8 == 0:
        ws = wsg(moe.MOEX_STAGE_TRAIN_BALANCED)
        y = torch.empty_like(x)
        moe.moe_forward_train(p, x, wr, bias, W1, W2, y, ws.t)
        run("backward balanced", {"dx": Guarded((T, d), BF), "dwr": Guarded((d, E), BF), "db": Guarded((E,), F32),
                                  "dW1": Guarded((E, d, de), BF), "dW2": Guarded((E, de, d), BF),
                                  "loss": Guarded((1,), F32), "c": Guarded((E,), i32), "mp": Guarded((E,), F32),
                                  "ws": ws},
            {"x": x, "wr": wr, "W1": W1, "W2": W2, "dy": dy, "mask": mask},
            lambda t: moe.moex_backward_balanced(p, x, wr, W1, W2, dy, mask, 0.1, t["dx"], t["dwr"], t["db"],
                                                 t["dW1"], t["dW2"], t["loss"], t["c"], t["mp"], t["ws"]))


def test_training_step_of_a_block(moe):
    """norm -> layer (training forward) -> layer backward with the balance loss ->
    norm backward, against the oracle's chain on the same rounded activations."""
    announce("block training step")
    T, d, E, k, de = 160, 256, 8, 2, 128
    cfg = scaled_config("fine_grained", T=T, d_model=d, E=E, k=k, d_expert=de, suffix="step")
    inp = make_inputs(cfg, seed=9, device="cuda")
    wr, W1, W2 = inp["w_router"], inp["W1"], inp["W2"]
    x, res, gain = randn((T, d), 1.0, BF, 1), randn((T, d), 1.0, BF, 2), (1 + 0.1 * randn((d,), 1.0, F32, 3)).to(BF)
    dy = make_dense((T, d), 1.0, seed=9, tag=9, device="cuda")
    p = moe.make_problem(T, d, E, k, de, BF)
    e = lambda shape, dt=BF: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    h, n, r, y, dn, dx, dg = e((T, d)), e((T, d)), e((T,), F32), e((T, d)), e((T, d)), e((T, d)), e((d,), F32)
    dwr, dW1, dW2, loss = e((d, E)), torch.empty_like(W1), torch.empty_like(W2), e((1,), F32)
    ws = e((moe.moex_workspace_size(p, moe.MOEX_STAGE_TRAIN_BALANCED),), torch.uint8)
    nws = e((moe.moex_workspace_size(p, moe.MOEX_STAGE_NORM_BACKWARD),), torch.uint8)
    moe.moex_add_rmsnorm(p, x, res, gain, 1e-6, h, n, None, None, r)
    moe.moe_forward_train(p, n, wr, None, W1, W2, y, ws)
    moe.moex_backward_balanced(p, n, wr, W1, W2, dy, None, 0.1, dn, dwr, None, dW1, dW2, loss, None, None, ws)
    moe.moex_add_rmsnorm_backward(p, h, gain, r, dn, dy, dx, dg, nws)  # the stream carries dy past the layer
    torch.cuda.synchronize()
    ref = oracle.backward(host_array(n), host_array(wr), None, host_array(W1), host_array(W2), k, "bf16",
                          host_array(dy))
    route = oracle.route(f64(n), f64(wr), None, k)
    bal = ob.balance_loss(route["logits"].astype(np.float64), route["idx"].astype(np.int64), None, 0.1)
    assert abs(float(loss) - bal["loss"]) <= 1e-5 * bal["loss"]
    dn_ref = ref["dx"] + bal["dlogits"] @ f64(wr).T
    dwr_ref = ref["dw_router"] + f64(n).T @ bal["dlogits"]
    assert rel_err(f64(dn), dn_ref) <= 1e-2 and rel_err(f64(dwr), dwr_ref) <= 1e-2
    assert rel_err(f64(dW1), ref["dW1"]) <= 1e-2 and rel_err(f64(dW2), ref["dW2"]) <= 1e-2
    dx_ref, dg_ref = ob.rmsnorm_backward(f64(h), f64(gain), f64(r), f64(dn), f64(dy))
    assert rel_err(f64(dx), dx_ref) <= 2.0 ** -8 and rel_err(f64(dg), dg_ref) <= 1e-5
