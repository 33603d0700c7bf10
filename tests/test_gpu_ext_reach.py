"""The operators around the layer past 2^31 elements, and captured into a graph."""

import numpy as np
import pytest
import torch

from ext_helpers import f64, gen, quantized, randn
from gpu_helpers import U32, announce, needs_gpu
from oracle import block_ops as ob

pytestmark = [pytest.mark.gpu, needs_gpu]

BF, F32 = torch.bfloat16, torch.float32


def test_norm_past_32_bits(moe):
    """2.2e9 elements: the last rows are those of a call on them alone, bit for bit."""
    announce("norm reach")
    T, d, n = 270000, 8192, 700
    p, q = moe.make_problem(T, d, 1, 1, 64, BF), moe.make_problem(n, d, 1, 1, 64, BF)
    tail = slice(T - n, T)
    x = torch.full((T, d), 0.5, dtype=BF, device="cuda")
    res = torch.full((T, d), 0.25, dtype=BF, device="cuda")
    x[tail], res[tail] = randn((n, d), 1.0, BF, 1), randn((n, d), 1.0, BF, 2)
    gain = randn((d,), 1.0, BF, 3)

    def run(p, x, res):
        h, y = torch.empty_like(x), torch.empty_like(x)
        y8 = torch.empty((p.T, ob.code_pitch(d)), dtype=torch.uint8, device="cuda")
        ys = torch.empty((p.T, ob.scale_pitch(d)), dtype=torch.uint8, device="cuda")
        r = torch.empty(p.T, dtype=F32, device="cuda")
        moe.moex_add_rmsnorm(p, x, res, gain, 1e-5, h, y, y8, ys, r)
        dx, dg = torch.empty_like(x), torch.empty(d, dtype=F32, device="cuda")
        ws = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_NORM_BACKWARD), dtype=torch.uint8, device="cuda")
        moe.moex_add_rmsnorm_backward(p, h, gain, r, x, res, dx, dg, ws)
        return h, y, y8, ys, r, dx

    big, small = run(p, x, res), run(q, x[tail].contiguous(), res[tail].contiguous())
    torch.cuda.synchronize()
    for a, b in zip(big, small):
        assert torch.equal(a[tail], b)
    assert bool((big[0][: T - n] == 0.75).all())  # and nothing else was hit
    assert torch.equal(big[1][0], big[1][T - n - 1])


def test_balance_past_32_bits(moe):
    """2.2e9 logits: counts exactly, means and the last rows' gradient against float64."""
    announce("balance reach")
    T, E, n = 8_400_000, 256, 50
    logits = torch.randn((T, E), generator=gen(4), device="cuda")
    idx = logits.argmax(dim=1).to(torch.int32).reshape(T, 1)
    p = moe.make_problem(T, 64, E, 1, 64, F32)
    loss, mean = torch.empty(1, device="cuda"), torch.empty(E, device="cuda")
    counts, dl = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty((T, E), device="cuda")
    ws = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_BALANCE), dtype=torch.uint8, device="cuda")
    moe.moex_balance_loss(p, logits, idx, None, 1.0, loss, counts, mean, dl, ws)
    torch.cuda.synchronize()
    assert torch.equal(counts.long(), torch.bincount(idx.reshape(-1).long(), minlength=E))
    P = torch.zeros(E, dtype=torch.float64, device="cuda")
    for t in range(0, T, 200_000):
        P += torch.softmax(logits[t:t + 200_000].double(), dim=1).sum(dim=0)
    P /= T
    # a float32 p is off by (E + 8) units at most, and a workgroup's 2051 rows are
    # added per token group, 129 at a time, in float32
    assert bool(((mean.double() - P).abs() <= (E + 8 + 129) * U32 * P).all())
    f = counts.double() / T
    assert abs(float(loss) - float(E * (f * P).sum())) <= (E + 8 + 130) * U32 * float(E * (f * P).sum())
    q = torch.softmax(logits[-n:].double(), dim=1)
    m = q.argmax(dim=1)
    g = f[None, :] - f[m][:, None]
    want = (E / T) * q * (g - (q * g).sum(dim=1, keepdim=True))
    size = (E / T) * q * (g.abs() + (q * g.abs()).sum(dim=1, keepdim=True))
    assert bool(((dl[-n:].double() - want).abs() <= (2 * E + 24) * U32 * size).all())


@pytest.mark.parametrize("tiles", ["0", "1"])
def test_experts_past_32_bits(moe, monkeypatch, tiles):
    """2.2e9 elements of y_perm: the last group's last rows are those of a call on them alone."""
    announce(f"experts reach tiles={tiles}")
    monkeypatch.setenv("MOE_FP8_TILES", tiles)
    T, d, E, k, de, n = 131500, 2048, 8, 8, 256, 300
    p = moe.make_problem(T, d, E, k, de, BF)
    W1, W2 = randn((E, d, de), 0.02, BF, 5), randn((E, de, d), 0.05, BF, 6)
    Q = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in moe.expert_shapes(p)]
    moe.moex_quantize_experts(p, W1, W2, *Q)
    x8, xs, _ = quantized(moe, randn((n, d), 1.0, BF, 7))

    def run(p, x8, xs, perm, off):
        y = torch.empty((p.T * p.k, d), dtype=BF, device="cuda")
        ws = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_FFN_FP8), dtype=torch.uint8, device="cuda")
        moe.moex_grouped_ffn_fp8(p, x8, xs, perm, off, *Q, y, ws)
        return y

    b8, bs = torch.empty((T, x8.shape[1]), dtype=torch.uint8, device="cuda"), torch.zeros((T, xs.shape[1]),
                                                                                        dtype=torch.uint8, device="cuda")
    b8.fill_(0x38)  # ones
    bs[:, : d // 128] = 120
    b8[-n:], bs[-n:] = x8, xs
    R = T * k
    perm = (torch.arange(R, device="cuda") % (T - n)).to(torch.int32)
    perm[-n:] = torch.arange(T - n, T, device="cuda", dtype=torch.int32)
    off = torch.tensor([R // E * e for e in range(E)] + [R], dtype=torch.int32, device="cuda")
    big = run(p, b8, bs, perm, off)
    q = moe.make_problem(n, d, E, 1, de, BF)
    small = run(q, x8, xs, torch.arange(n, device="cuda", dtype=torch.int32),
                torch.tensor([0] * E + [n], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(big[-n:], small)
    assert torch.equal(big[0], big[R // E - 1])


def test_training_operators_replay(moe):
    """Norm forward and backward and the balance loss in one captured graph, replayed
    on new inputs with eager work of the same kind between the replays."""
    announce("training replay")
    T, d, E, k = 1500, 320, 24, 3
    p = moe.make_problem(T, d, E, k, 64, BF)
    x, res, dy = (torch.empty((T, d), dtype=BF, device="cuda") for _ in range(3))
    gain = randn((d,), 1.0, BF, 8)
    lg, ix = torch.empty((T, E), device="cuda"), torch.empty((T, k), dtype=torch.int32, device="cuda")
    mk = torch.empty(T, dtype=torch.bool, device="cuda")
    wsn = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_NORM_BACKWARD), dtype=torch.uint8, device="cuda")
    wsb = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_BALANCE), dtype=torch.uint8, device="cuda")

    def outputs():
        new = lambda s, dt: torch.full(s, 7, dtype=dt, device="cuda")  # noqa: E731
        return [new((T, d), BF), new((T, d), BF), new((T,), F32), new((T, d), BF), new((d,), F32), new((1,), F32),
                new((E,), torch.int32), new((E,), F32), new((T, E), F32)]

    def fill(seed):
        for i, t in enumerate((x, res, dy)):
            t.copy_(randn((T, d), 1.0, BF, seed + i))
        lg.copy_(randn((T, E), 1.0, F32, seed + 3))
        ix.copy_(torch.sort(lg, dim=1, descending=True).indices[:, :k].to(torch.int32))
        mk.copy_(torch.rand((T,), generator=gen(seed + 4), device="cuda") < 0.8)

    def run(o):
        moe.moex_add_rmsnorm(p, x, res, gain, 1e-5, o[0], o[1], None, None, o[2])
        moe.moex_balance_loss(p, lg, ix, mk, 0.01, o[5], o[6], o[7], o[8], wsb)
        moe.moex_add_rmsnorm_backward(p, o[0], gain, o[2], dy, None, o[3], o[4], wsn)

    out, eager = outputs(), outputs()
    fill(10)
    run(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for seed in (20, 30, 40, 50):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        run(eager)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
    assert np.isfinite(f64(out[3])).all()
