"""The float64 forms of the operators around the layer, pinned to closed forms,
torch's own conversions and differences (CPU only)."""

import math

import numpy as np
import pytest
import torch

from oracle import block_ops as ob


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(ob.E4M3))
    assert np.array_equal(t[~np.isnan(t)], ob.E4M3[~np.isnan(t)])
    assert ob.E4M3[0x7E] == 448.0 and ob.E4M3[1] == 2.0 ** -9


def test_round_e4m3_is_torchs_on_float32():
    g = np.random.default_rng(0)
    v = np.concatenate([g.normal(size=20000) * 2.0 ** g.integers(-12, 9, 20000), [0.0, -0.0, 448.0, -448.0, 2.0 ** -10,
                        3 * 2.0 ** -10, 17.0, 18.0, 19.0, 460.0, 464.0]]).astype(np.float32)
    v = v[np.abs(v) <= 464]
    t = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ob.round_e4m3(v.astype(np.float64)), t)
    assert set(ob.round_e4m3(np.array([np.inf, np.nan, 500.0])) & 127) == {127}


def test_block_exponent_is_the_smallest_that_fits():
    g = np.random.default_rng(1)
    a = np.concatenate([2.0 ** g.uniform(-100, 100, 2000), 448.0 * 2.0 ** np.arange(-60, 60)])
    e = ob.block_exponent(a)
    assert np.all(a <= 448.0 * 2.0 ** e) and np.all(a > 448.0 * 2.0 ** (e - 1.0))
    assert ob.block_exponent(np.array([0.0, 1e-45, np.inf, 3.4e38])).tolist() == [-120, -120, 120, 120]


def test_encode_decode_error_is_half_a_step():
    g = np.random.default_rng(2)
    v = g.normal(size=(5, 320))
    c, e = ob.encode(v)
    assert c.shape == (5, 384) and e.shape == (5, 3) and not c[:, 320:].any()
    d = ob.decode(c, e)[:, :320]
    step = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * np.repeat(2.0 ** e, 128, axis=1)[:, :320])
    assert np.all(np.abs(d - v) <= step)


def test_weight_layout_places_every_code():
    g = np.random.default_rng(3)
    w = g.normal(size=(2, 192, 64))
    q, s, dec = ob.weight_layout(w)
    assert q.shape == (2, 2, 2, 4, 2, 32, 16) and s.shape == (2, 2, 2, 32)
    for e, k, n in ((0, 0, 0), (1, 191, 63), (0, 130, 33), (1, 77, 31)):
        kb, r = divmod(k, 128)
        code = q[e, n // 32, kb, r // 32, r % 32 // 16, n % 32, r % 16]
        assert ob.E4M3[code] * 2.0 ** (int(s[e, n // 32, kb, n % 32]) - 127) == dec[e, k, n]
    assert np.all(np.abs(dec[:, :192] - w) <= 0.07 * np.abs(w).max())
    assert not dec[:, 192:].any()


def test_rmsnorm_backward_is_the_difference_quotient():
    g = np.random.default_rng(4)
    h, gain, dy, dh = g.normal(size=(3, 64)), g.normal(size=64), g.normal(size=(3, 64)), g.normal(size=(3, 64))
    loss = lambda hh, gg: float((ob.rmsnorm(hh, gg, 1e-3)[0] * dy).sum() + (hh * dh).sum())  # noqa: E731
    r = ob.rmsnorm(h, gain, 1e-3)[1]
    dx, dg = ob.rmsnorm_backward(h, gain, r, dy, dh)
    for i, j in ((0, 0), (2, 63), (1, 17)):
        s = 1e-6
        up, dn = h.copy(), h.copy()
        up[i, j] += s
        dn[i, j] -= s
        assert abs((loss(up, gain) - loss(dn, gain)) / (2 * s) - dx[i, j]) < 1e-7 * (1 + abs(dx[i, j])) * 100
        gu, gd = gain.copy(), gain.copy()
        gu[j] += s
        gd[j] -= s
        assert abs((loss(h, gu) - loss(h, gd)) / (2 * s) - dg[j]) < 1e-5


def test_balance_gradient_is_the_difference_quotient_and_even_routing_has_none():
    g = np.random.default_rng(5)
    T, E, k = 7, 6, 2
    logits = g.normal(size=(T, E))
    idx = np.argsort(-logits, axis=1)[:, :k]
    mask = np.array([1, 1, 0, 1, 1, 1, 0])
    out = ob.balance_loss(logits, idx, mask, 0.3)
    assert out["counts"].sum() == 5 * k and not out["dlogits"][mask == 0].any()
    for t, e in ((0, 0), (3, 5), (2, 1)):
        s = 1e-6
        up, dn = logits.copy(), logits.copy()
        up[t, e] += s
        dn[t, e] -= s
        num = (ob.balance_loss(up, idx, mask, 0.3)["loss"] - ob.balance_loss(dn, idx, mask, 0.3)["loss"]) / (2 * s)
        assert abs(num - out["dlogits"][t, e]) < 1e-8
    # every expert chosen equally often: the loss is coef, its least value for even probabilities, the gradient 0
    even = np.array([[0, 1], [2, 3], [4, 5]])
    o = ob.balance_loss(np.zeros((3, 6)), even, None, 0.25)
    assert abs(o["loss"] - 0.25) < 1e-15 and np.abs(o["dlogits"]).max() < 1e-17
    assert ob.balance_loss(logits, idx, np.zeros(T), 1.0)["loss"] == 0.0


@pytest.mark.parametrize("E", [1, 3])
def test_grouped_ffn_fp8_of_exact_values_is_the_float_ffn(E):
    """Weights and rows that e4m3 holds exactly: the first product is exact, and
    the result differs from the unquantised FFN by the hidden values' rounding."""
    g = np.random.default_rng(6)
    x = g.integers(-3, 4, size=(6, 128)).astype(float)
    w1, w2 = g.integers(-2, 3, size=(E, 128, 128)) / 16.0, g.integers(-2, 3, size=(E, 128, 64)) / 8.0
    off = np.linspace(0, 6, E + 1).astype(int)
    y = ob.grouped_ffn_fp8(x, off, w1, w2)
    for e in range(E):
        h = ob.gelu_tanh(x[off[e]:off[e + 1]] @ w1[e])
        ref = h @ w2[e]
        assert np.all(np.abs(y[off[e]:off[e + 1]] - ref) <= (2.0 ** -4 * np.abs(h) + 2.0 ** -10) @ np.abs(w2[e]) + 1e-12)
