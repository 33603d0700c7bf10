"""The float64 forms of what trains the layer's surroundings, pinned to torch's own
optimizer, autograd and conversions, to differences and to counts (CPU only)."""

import math

import numpy as np
import pytest
import torch

from oracle import train_ops as to


def test_dispatch_index_by_hand():
    idx = np.array([[2, 0], [0, 0], [-1, 2], [5, 1]])
    i = to.dispatch_index(idx, 3)
    assert i["counts"].tolist() == [3, 1, 2] and i["offsets"].tolist() == [0, 3, 4, 6]
    assert i["perm"].tolist() == [0, 1, 1, 3, 0, 2]
    assert i["inv"].tolist() == [4, 0, 1, 2, -1, 5, -1, 3]


def test_ways_and_gradients_are_autograds():
    g = np.random.default_rng(0)
    T, k, E, d = 9, 3, 4, 5
    idx = g.integers(-1, E + 1, (T, k))
    i = to.dispatch_index(idx, E)
    x, w, add = (torch.from_numpy(g.normal(size=s)).requires_grad_() for s in ((T, d), (T, k), (T, d)))
    sel = torch.from_numpy(i["order"])
    rows = x[sel // k] * w.reshape(-1)[sel][:, None]
    assert np.allclose(rows.detach().numpy(), to.to_rows(x.detach().numpy(), i, w.detach().numpy()), atol=1e-14)
    dr = g.normal(size=rows.shape)
    rows.backward(torch.from_numpy(dr))
    assert np.allclose(x.grad.numpy(), to.from_rows(dr, i, w.detach().numpy(), None, T), atol=1e-14)
    assert np.allclose(w.grad.numpy(), to.dots(dr, x.detach().numpy(), i, k), atol=1e-14)
    w.grad = None
    y_perm = torch.from_numpy(g.normal(size=(i["perm"].size, d))).requires_grad_()
    y = add + torch.zeros(T, d, dtype=torch.float64).index_add(0, sel // k, y_perm * w.reshape(-1)[sel][:, None])
    ref = to.from_rows(y_perm.detach().numpy(), i, w.detach().numpy(), add.detach().numpy(), T)
    assert np.allclose(y.detach().numpy(), ref, atol=1e-14)
    dy = g.normal(size=(T, d))
    y.backward(torch.from_numpy(dy))
    assert np.allclose(y_perm.grad.numpy(), to.to_rows(dy, i, w.detach().numpy()), atol=1e-14)
    assert np.allclose(w.grad.numpy(), to.dots(y_perm.detach().numpy(), dy, i, k), atol=1e-14)
    assert np.array_equal(add.grad.numpy(), dy)


def test_gate_backward_is_autograds():
    g = np.random.default_rng(1)
    lg = torch.from_numpy(g.normal(size=(6, 7))).requires_grad_()
    idx = np.stack([g.permutation(7)[:3] for _ in range(6)])
    dg, add = g.normal(size=(6, 3)), g.normal(size=(6, 7))
    torch.softmax(lg, 1).gather(1, torch.from_numpy(idx)).backward(torch.from_numpy(dg))
    assert np.allclose(lg.grad.numpy() + add, to.gate_backward(lg.detach().numpy(), idx, dg, add), atol=1e-14)
    empty = np.full((1, 4), -np.inf)
    assert np.array_equal(to.gate_backward(empty, np.array([[1]]), np.ones((1, 1)), None), np.zeros((1, 4)))


@pytest.mark.parametrize("name", ["none", "gelu", "silu", "relu"])
def test_activations_are_torchs(name):
    u = torch.linspace(-9, 9, 1801, dtype=torch.float64).requires_grad_()
    f = {"none": lambda v: v, "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
         "silu": torch.nn.functional.silu, "relu": torch.relu}[name]
    f(u).sum().backward()
    assert np.allclose(to.act(u.detach().numpy(), name), f(u).detach().numpy(), atol=1e-13)
    assert np.allclose(to.act_slope(u.detach().numpy(), name), u.grad.numpy(), atol=1e-13)


def test_adamw_is_torchs():
    g = np.random.default_rng(2)
    p = torch.nn.Parameter(torch.from_numpy(g.normal(size=50)))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        gr = g.normal(size=50)
        p.grad = torch.from_numpy(gr)
        opt.step()
        q, m, v = to.adamw(q, gr, m, v, t, 1e-2, 0.8, 0.95, 1e-6, 0.1)
        assert np.allclose(p.detach().numpy(), q, rtol=1e-12, atol=1e-14)


def test_code_tables_are_torchs():
    c = torch.arange(124, dtype=torch.uint8)
    assert np.array_equal(to.E5M2_POS, c.view(torch.float8_e5m2).double().numpy())
    assert to.E5M2_POS[-1] == 57344 and to.E4M3_POS[-1] == 448


@pytest.mark.parametrize("table,keep", [(to.E4M3_POS, False), (to.E5M2_POS, True)], ids=["m", "v"])
def test_rounding_is_unbiased_and_stays_between_neighbours(table, keep):
    x = np.repeat([0.3, 1.0, 100.0, 1.7, 0.011, 448.0 if not keep else 57344.0], 1)
    total = np.zeros(x.size)
    N = 4096
    for r in range(0, 65536, 65536 // N):
        codes, e = to.round_stochastic(x, np.full(x.size, r), table, keep)
        v = to.decode(codes, e, table)
        s = np.ldexp(1.0, int(e[0]))
        assert np.all(np.abs(v - x) < np.maximum(x * 2.0 ** -(2 if keep else 3), table[1] * s) + 1e-12)
        total += v
    # the mean over all random numbers is x, within one of N parts of a spacing
    assert np.all(np.abs(total / N - x) <= x * 2.0 ** -(2 if keep else 3) / N * 1.01 + table[1] * s / N)


def test_rounding_edges():
    zero = np.zeros(128)
    c, e = to.round_stochastic(zero, np.full(128, 65535), to.E5M2_POS, True)
    assert not c.any() and e.tolist() == [-120]
    x = zero.copy()
    x[0], x[1] = 1.0, 1e-30
    c, _ = to.round_stochastic(x, np.zeros(128), to.E5M2_POS, True)
    assert c[1] == 1 and c[2] == 0  # a second moment that is not 0 stays so
    c, _ = to.round_stochastic(x, np.zeros(128), to.E4M3_POS, False)
    assert c[1] == 0
    x[2], x[3] = np.nan, np.inf
    c, e = to.round_stochastic(x, np.zeros(128), to.E4M3_POS, False)
    assert c[2] == 127 and c[3] == 127 and e.tolist() == [120]


def test_draws_are_spread():
    r = to.draws(20000, 7, 3, 1)
    for half in (r & 0xFFFF, r >> 16):
        n = np.bincount(half >> 12, minlength=16)  # 16 cells of 1250: standard deviation 34
        assert np.all(np.abs(n - 1250) < 5 * 34)
    assert abs(np.corrcoef(r & 0xFFFF, r >> 16)[0, 1]) < 5 / math.sqrt(20000)
    assert to.draws(1, 7, 3, 1, first=5)[0] == r[5] and to.draws(1, 7, 3, 1, first=(1 << 32) + 5)[0] != r[5]
    assert to.draws(4, 7, 4, 1).tolist() != r[:4].tolist() != to.draws(4, 7, 3, 2).tolist()
