"""The optimizer's step on the GPU, against float64.

Moments and codes are compared bit for bit: both sides take the same products and sums
in 64 bits, each rounded once. A parameter's move is made in float32 from a root and a
reciprocal of one unit each, the moments rounded to float32, and four more roundings:
within 2^-20 of itself; the parameter is rounded twice.
"""

import numpy as np
import pytest
import torch

from ext_helpers import assert_within, gen
from gpu_helpers import U32, announce, f64, needs_gpu
from oracle import train_ops as to
from test_gpu_canary import Guarded

pytestmark = [pytest.mark.gpu, needs_gpu]

BF, F32 = torch.bfloat16, torch.float32
LR, B1, B2, EPS, WD = 1e-2, 0.9, 0.99, 1e-8, 0.1


def params_of(sizes, seed):
    """(param, gradient) pairs: sizes of (n, parameter type, gradient type)."""
    g = gen(seed)
    out = []
    for n, pt, gt in sizes:
        scale = torch.exp2(3 * torch.randn(((n + 127) // 128, 1), generator=g, device="cuda") - 6)
        gr = (torch.randn(((n + 127) // 128, 128), generator=g, device="cuda") * scale).reshape(-1)[:n].contiguous()
        out.append(((torch.randn(n, generator=g, device="cuda") * 0.1).to(pt), gr.to(gt)))
    return [p for p, _ in out], [g for _, g in out]


class Mirror:
    """The same steps in float64, from the optimizer's own state before each."""

    def __init__(self, opt):
        self.opt = opt
        self.t = int(opt.counter[0])

    def before(self):
        o = self.opt
        self.p = [f64(p if m is None else m) for p, m in zip(o.params, o.master)]
        self.m, self.v = [], []
        for m, ms, v, vs in zip(o.m, o.m_scale, o.v, o.v_scale):
            if ms is None:
                self.m.append(f64(m))
                self.v.append(f64(v))
                continue
            for dst, c, s, tab in ((self.m, m, ms, to.E4M3_POS), (self.v, v, vs, to.E5M2_POS)):
                dst.append(to.decode(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy().astype(np.int64) - 127, tab))

    def check(self, grads, lr=LR, scale=1.0, wd=WD, random=True):
        torch.cuda.synchronize()
        o, self.t = self.opt, self.t + 1
        assert o.counter.tolist() == [self.t, 0]
        for j, gr in enumerate(grads):
            g = f64(gr) * np.float64(scale)
            p, m, v = to.adamw(self.p[j], g, self.m[j], self.v[j], self.t, lr, B1, B2, EPS, wd)
            m = B1 * self.m[j] + (1 - B1) * g
            v = B2 * self.v[j] + ((1 - B2) * g) * g  # the order of the products
            got = f64(o.params[j] if o.master[j] is None else o.master[j])
            move = np.abs(p - self.p[j])
            assert_within(f"param {j}", got, p, 2.0 ** -20 * move + 2 * U32 * (np.abs(p) + np.abs(self.p[j])))
            if o.master[j] is not None:
                assert torch.equal(o.params[j], o.master[j].to(BF).view_as(o.params[j]))
            if o.m_scale[j] is None:
                for name, x, y in (("m", o.m[j], m), ("v", o.v[j], v)):
                    same = x.cpu().numpy() == y.astype(np.float32)
                    assert same.all(), (name, j, int((~same).sum()))
            elif random:
                r = to.draws(g.size, o.seed, self.t, j)
                for name, x, rr, c, s, tab in (("m", m, r & 0xFFFF, o.m[j], o.m_scale[j], to.E4M3_POS),
                                               ("v", v, r >> 16, o.v[j], o.v_scale[j], to.E5M2_POS)):
                    codes, e = to.round_stochastic(x, rr, tab, name == "v")
                    assert (s.cpu().numpy().astype(np.int64) - 127 == e).all(), (name, j)
                    same = c.view(torch.uint8).cpu().numpy() == codes
                    assert same.all(), (name, j, int((~same).sum()))


SIZES = [(1, BF, BF), (7, F32, F32), (128, BF, F32), (129, F32, BF), (2047, BF, BF), (2048, F32, F32), (2049, BF, BF),
         (4100, BF, F32), (10000, F32, BF)]


@pytest.mark.parametrize("bits", [32, 8])
def test_against_float64(moe, bits):
    announce(f"adamw bits={bits}")
    params, grads = params_of(SIZES, 1)
    opt = moe.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, bits=[bits] * len(params), seed=3)
    ref = Mirror(opt)
    for step in range(3):
        grads = [g * (1 + step) for g in grads]
        ref.before()
        opt.step(grads)
        ref.check(grads)


def test_mixed_moments_factors_and_many_tensors(moe):
    """Lists of more than one launch, with moments of both kinds, factors and decays of their own."""
    announce("adamw 130 tensors")
    n = 130
    params, grads = params_of([(100 + 37 * i, BF if i % 3 else F32, BF if i % 2 else F32) for i in range(n)], 2)
    bits = [8 if i % 2 else 32 for i in range(n)]
    factor, decay = [1.0 + i % 4 for i in range(n)], [0.1 * (i % 3) for i in range(n)]
    opt = moe.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decay, lr_factor=factor, bits=bits, max_norm=1e9)
    ref = Mirror(opt)
    ref.before()
    norm = opt.step(grads)
    torch.cuda.synchronize()
    total = np.sqrt(sum(np.sum(f64(g) ** 2) for g in grads))
    assert abs(float(norm) - total) <= 2 * U32 * total
    before, t = (ref.p, ref.m, ref.v), ref.t
    for i in range(n):  # one at a time: each has its own lr and decay
        p, m, v = to.adamw(before[0][i], f64(grads[i]), before[1][i], before[2][i], t + 1, LR * factor[i], B1, B2, EPS, decay[i])
        got = f64(params[i] if opt.master[i] is None else opt.master[i])
        assert_within(f"param {i}", got, p, 2.0 ** -20 * np.abs(p - before[0][i]) + 2 * U32 * (np.abs(p) + np.abs(before[0][i])))
        if bits[i] == 8:
            codes, e = to.round_stochastic(m, to.draws(m.size, 0, t + 1, i) & 0xFFFF, to.E4M3_POS, False)
            assert np.array_equal(opt.m[i].view(torch.uint8).cpu().numpy(), codes)
    assert opt.counter.tolist() == [1, 0]


@pytest.mark.parametrize("max_norm,clips", [(0.5, True), (1e6, False), (float("inf"), False)])
def test_clipping(moe, max_norm, clips):
    announce(f"adamw max_norm={max_norm}")
    params, grads = params_of([(5000, BF, BF), (33, F32, F32)], 3)
    total = np.sqrt(sum(np.sum(f64(g) ** 2) for g in grads))
    opt = moe.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, bits=8, max_norm=max_norm)
    ref = Mirror(opt)
    ref.before()
    norm = float(opt.step(grads))
    assert abs(norm - total) <= 2 * U32 * total
    scale = float(opt.scale)
    assert scale == (float(np.float32(max_norm / total)) if clips else 1.0) or abs(scale - max_norm / total) <= U32 * scale
    ref.check(grads, scale=np.float32(scale))


def test_clipped_is_norm_and_step(moe):
    """One call and two give the same bits: norm, factor, parameters and moments, also of long lists."""
    announce("adamw clipped in one call and in two")
    params, grads = params_of([(300 + 91 * i, BF if i % 2 else F32, BF) for i in range(140)], 14)
    other = [p.clone() for p in params]
    mk = lambda ps: moe.AdamW(ps, lr=LR, bits=[8 if i % 3 else 32 for i in range(140)], max_norm=0.3, seed=2)  # noqa: E731
    a, b = mk(params), mk(other)
    a.step(grads)
    norm, scale = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    ws = torch.empty(moe.MOET_GRAD_NORM_WS_BYTES, dtype=torch.uint8, device="cuda")
    for e, g in zip(b._entries, grads):
        moe.set_grad(e, g, 0)
    moe.moet_grad_norm(b._list, 0.3, norm, scale, ws)
    moe.moet_adamw(b._list, moe.AdamWOptions(LR, 0.9, 0.999, 1e-8, 2), b.counter, None, scale)
    torch.cuda.synchronize()
    assert torch.equal(norm, a.norm) and torch.equal(scale, a.scale) and float(scale) < 1
    for x, y in zip((*params, *a.m, *a.v, a.counter), (*other, *b.m, *b.v, b.counter)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_gradients_that_are_not_finite_leave_the_step_out(moe, bad):
    announce(f"adamw skips {bad}")
    params, grads = params_of([(5000, BF, BF), (33, F32, F32)], 4)
    opt = moe.AdamW(params, bits=8, max_norm=1.0)
    opt.step(grads)
    everything = [t for t in (*params, *opt.master, *opt.m, *opt.v, *opt.m_scale, *opt.v_scale, opt.counter) if t is not None]
    before = [t.clone() for t in everything]
    grads[0][4321] = bad
    opt.step(grads)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(everything, before))
    assert torch.isnan(opt.scale).item()
    grads[0][4321] = 0.0
    opt.step(grads)
    assert opt.counter.tolist() == [2, 0]


def test_without_clipping_only_the_values_touched_are_lost(moe):
    announce("adamw NaN without clipping")
    params, grads = params_of([(5000, F32, F32)], 5)
    grads[0][100], grads[0][3000] = float("nan"), float("inf")
    for bits in (8, 32):
        opt = moe.AdamW([params[0].clone()], bits=[bits])
        opt.step(grads)
        m, v = opt.m[0].float(), opt.v[0].float()
        bad = torch.zeros(5000, dtype=torch.bool, device="cuda")
        bad[100] = bad[3000] = True
        assert torch.equal(~torch.isfinite(m), bad) and torch.equal(~torch.isfinite(v), bad)
        assert torch.equal(~torch.isfinite(opt.params[0]), bad)


def test_zero_gradients(moe):
    """Moments of zeros stay zeros and move nothing but the decay."""
    announce("adamw zeros")
    p = torch.full((3000,), 2.0, device="cuda")
    for bits in (8, 32):
        q = p.clone()
        opt = moe.AdamW([q], lr=0.5, weight_decay=0.25, bits=[bits], max_norm=1.0)
        norm = opt.step([torch.zeros_like(p)])
        torch.cuda.synchronize()
        assert float(norm) == 0.0 and bool((q == 2.0 - 0.5 * 0.25 * 2.0).all())
        assert not opt.m[0].float().any() and not opt.v[0].float().any()


def test_beta_zero_and_factors_of_lr(moe):
    announce("adamw betas 0, lr_scale")
    params, grads = params_of([(300, F32, F32)], 6)
    before = f64(params[0])
    opt = moe.AdamW(params, lr=0.1, betas=(0.0, 0.0), eps=1e-6, weight_decay=0.0)
    opt.lr_scale.fill_(0.5)
    opt.step(grads)
    g = f64(grads[0])
    want = before - 0.05 * g / (np.abs(g) + 1e-6)
    assert_within("param", f64(params[0]), want, 2.0 ** -20 * 0.05 + 2 * U32 * np.abs(before))


def test_second_moment_stays_above_zero(moe):
    """Values 2^-40 of their block's largest: m may round to a step, v must not vanish under it."""
    announce("adamw floor of v")
    g = torch.full((128,), 2.0 ** -20, device="cuda")
    g[0] = 2.0 ** 20
    p = torch.zeros(128, device="cuda")
    opt = moe.AdamW([p], lr=1.0, betas=(0.9, 0.999), eps=1e-15, weight_decay=0.0, bits=[8])
    for _ in range(5):
        opt.step([g])
        g = torch.zeros_like(g)
    torch.cuda.synchronize()
    assert bool((opt.v[0].float() > 0).all())
    # |m| is at most a step of its codes, 2^-9 of 2^(17 - 8 + ..), v at least one of its own: bounded moves
    assert bool((p.abs() < 100).all())


def test_unaligned_tails_and_guards(moe):
    """Nothing past a tensor's end is written, whatever its length."""
    announce("adamw guarded")
    for n in (1, 5, 127, 130, 2049, 4093):
        for bits in (8, 32):
            g = {"param": Guarded((n,), BF), "master": Guarded((n,), F32), "m": Guarded((n,), torch.float8_e4m3fn if bits == 8 else F32),
                 "v": Guarded((n,), torch.float8_e5m2 if bits == 8 else F32), "counter": Guarded((2,), torch.int32)}
            if bits == 8:
                g["m_scale"], g["v_scale"] = (Guarded(((n + 127) // 128,), torch.uint8) for _ in range(2))
            for k, v in g.items():
                v.t.view(torch.uint8).zero_()
                if k.endswith("_scale"):
                    v.t.fill_(7)
            state = {k: [g[k].t if k in g else None] for k in ("master", "m", "m_scale", "v", "v_scale")}
            opt = moe.AdamW([g["param"].t], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, bits=[bits],
                            state={**state, "counter": g["counter"].t}, seed=9)
            ref = Mirror(opt)
            _, grads = params_of([(n, BF, BF)], 7)
            ref.before()
            opt.step(grads)
            ref.check(grads)
            assert all(v.intact() for v in g.values()), (n, bits)


def test_empty_tensors_are_left_out(moe):
    announce("adamw empty tensor")
    params, grads = params_of([(600, F32, F32)], 8)
    a, b = params[0].clone(), params[0].clone()
    opt = moe.AdamW([a], lr=LR)
    opt.step(grads)
    e = moe.Tensor(n=0, lr_factor=1.0)
    st = [torch.zeros(600, device="cuda") for _ in range(2)]
    one = moe.tensor_entry(b, grads[0], None, st[0], None, st[1], None, 1.0, 0.01)
    counter = torch.zeros(2, dtype=torch.int32, device="cuda")
    norm, ws = torch.zeros(1, device="cuda"), torch.empty(moe.MOET_GRAD_NORM_WS_BYTES, dtype=torch.uint8, device="cuda")
    moe.moet_adamw([e, one, e], moe.AdamWOptions(LR, 0.9, 0.999, 1e-8, 0), counter, None, None)
    moe.moet_grad_norm([e, one, e], 1.0, norm, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and counter.tolist() == [1, 0]
    total = np.sqrt(np.sum(f64(grads[0]) ** 2))
    assert abs(float(norm) - total) <= 2 * U32 * total
    moe.moet_grad_norm([], 1.0, norm, None, ws)
    moe.moet_adamw([], moe.AdamWOptions(LR, 0.9, 0.999, 1e-8, 0), counter, None, None)
    torch.cuda.synchronize()
    assert float(norm) == 0.0 and counter.tolist() == [2, 0]


def test_state_goes_on_elsewhere(moe):
    """Steps from cloned buffers give the bits of the steps that were not interrupted."""
    announce("adamw resumed")
    params, grads = params_of([(5000, BF, BF), (300, F32, F32)], 9)
    a = moe.AdamW(params, lr=LR, bits=8, seed=5, max_norm=1.0)
    for _ in range(2):
        a.step(grads)
    torch.cuda.synchronize()
    clone = {k: [None if t is None else t.clone() for t in v] if isinstance(v, list) else v.clone() for k, v in a.state.items()}
    other = [p.clone() for p in params]
    b = moe.AdamW(other, lr=LR, bits=8, seed=5, max_norm=1.0, state=clone)
    for o in (a, b):
        o.step(grads)
    torch.cuda.synchronize()
    for x, y in zip((*params, *a.m, *a.v, a.counter), (*other, *b.m, *b.v, b.counter)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_graph_replays(moe):
    """Replays take the step number from the GPU: the bits of as many eager steps."""
    announce("adamw captured")
    params, grads = params_of([(70000, BF, BF), (300, F32, F32)], 10)
    mk = lambda ps: moe.AdamW(ps, lr=LR, bits=8, seed=6, max_norm=1.0)  # noqa: E731
    other = [p.clone() for p in params]
    a, b = mk(params), mk(other)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(grads)
    for i in range(4):
        for o in (a, b):
            o.lr_scale.fill_(1.0 - 0.2 * i)
        g.replay()
        b.step(grads)
        torch.cuda.synchronize()
        torch.randn(1000, device="cuda").sum().item()
        for x, y in zip((*params, *a.m, *a.v, a.counter, a.norm), (*other, *b.m, *b.v, b.counter, b.norm)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), i


def test_streams(moe):
    """Two optimizers at once; one made on a busy stream and used on another."""
    announce("adamw streams")
    params, grads = params_of([(200000, BF, BF), (300, F32, F32)], 11)
    copies = [[p.clone() for p in params] for _ in range(3)]
    opts = []
    side = [torch.cuda.Stream() for _ in range(3)]
    for ps, s in zip(copies, side):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(200_000_000)
            opts.append(moe.AdamW(ps, bits=8, seed=1, max_norm=1.0))
    for o, s in zip(opts, side[1:] + side[:1]):
        for _ in range(3):
            o.step(grads, s)
    for s in side:
        s.synchronize()
    for o, ps in zip(opts[1:], copies[1:]):
        assert all(torch.equal(x, y) for x, y in zip(ps, copies[0]))
        assert torch.equal(o.counter, opts[0].counter)


def test_past_32_bits(moe):
    """2^32 values and more: the last blocks' moments and draws."""
    n = (1 << 32) + 5000
    announce("adamw past 2^32 values")
    p = torch.zeros(n, dtype=BF, device="cuda")
    g = torch.zeros(n, dtype=BF, device="cuda")
    tail = 4096
    g[-tail:] = torch.randn(tail, generator=gen(12), device="cuda").to(BF)
    opt = moe.AdamW([p], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, bits=[8], max_norm=1e9, seed=8)
    norm = opt.step([g])
    torch.cuda.synchronize()
    x = f64(g[-tail:])
    assert abs(float(norm) - np.linalg.norm(x)) <= 2 * U32 * np.linalg.norm(x)
    first = (n - tail + 127) // 128 * 128  # whole blocks
    x = f64(g[first:])
    r = to.draws(n - first, 8, 1, 0, first=first)
    codes, e = to.round_stochastic((1 - B1) * x, r & 0xFFFF, to.E4M3_POS, False)
    assert np.array_equal(opt.m[0][first:].view(torch.uint8).cpu().numpy(), codes)
    codes, e = to.round_stochastic(((1 - B2) * x) * x, r >> 16, to.E5M2_POS, True)
    assert np.array_equal(opt.v[0][first:].view(torch.uint8).cpu().numpy(), codes)
    want = to.adamw(0 * x, x, 0 * x, 0 * x, 1, LR, B1, B2, EPS, WD)[0]
    assert_within("param", f64(opt.master[0][first:]), want, 2.0 ** -20 * np.abs(want))
    assert not p[:1 << 20].any()


def test_refusals(moe):
    params, grads = params_of([(300, F32, F32)], 13)
    opt = moe.AdamW(params)
    with pytest.raises(ValueError):
        opt.step([])
    with pytest.raises(ValueError, match="holds"):
        opt.step([grads[0][:100]])
    with pytest.raises(TypeError):
        opt.step([grads[0].half()])
    with pytest.raises(ValueError, match="contiguous"):
        opt.step([torch.randn(600, device="cuda")[::2]])
    with pytest.raises(moe.MoEError):
        opt.step([opt.m[0]])  # a gradient that is a moment
    with pytest.raises(ValueError, match="8 or in 32"):
        moe.AdamW(params, bits=16)
    with pytest.raises(ValueError, match="state needs"):
        moe.AdamW(params, state={"m": []})
    with pytest.raises(ValueError, match="max_norm"):
        moe.AdamW(params, max_norm=0.0)
    with pytest.raises(TypeError):
        moe.AdamW([params[0].half()])
