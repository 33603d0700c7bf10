"""RMS norm with residual and 8-bit rows, forward and backward, against float64."""

import numpy as np
import pytest
import torch

from ext_helpers import HALF, TINY, assert_within, codes_of, f64, randn
from gpu_helpers import U32, announce, needs_gpu
from oracle import block_ops as ob

pytestmark = [pytest.mark.gpu, needs_gpu]

BF, F32 = torch.bfloat16, torch.float32
CP, SP = ob.code_pitch, ob.scale_pitch

SHAPES = [  # T, d: every number of threads per row, half blocks at the end, single rows, ragged row groups
    (1, 64), (3, 64), (5, 128), (1, 320), (777, 320), (9, 512), (7, 576), (2, 1024), (33, 1088), (6, 2048), (3, 2112),
    (5, 4096), (3, 4160), (1, 7168), (2, 8192), (3, 8256), (1, 16384), (2, 16448), (2, 32768),
]


def forward(moe, x, res, gain, eps, y=True, q=True, stream=None):
    T, d = x.shape
    p = moe.make_problem(T, d, 1, 1, 64, x.dtype)
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    o = {"h": new((T, d), x.dtype) if res is not None else None, "y": new((T, d), x.dtype) if y else None,
         "y8": new((T, CP(d)), torch.float8_e4m3fn) if q else None,
         "scale": new((T, SP(d)), torch.uint8) if q else None, "rstd": new((T,), F32)}
    moe.moex_add_rmsnorm(p, x, res, gain, eps, o["h"], o["y"], o["y8"], o["scale"], o["rstd"], stream)
    return o


def check_forward(x, res, gain, eps, o):
    dt = x.dtype
    if res is not None:
        # one float32 addition of two exact values, rounded to the type as torch rounds
        h = (x.float() + res.float()).to(dt)
        assert torch.equal(o["h"], h)
    else:
        h = x
    h64, g64 = f64(h), f64(gain)
    y, r = ob.rmsnorm(h64, g64, float(np.float32(eps)))
    # r: one rounding to float32 of a float64 value that is off by far less
    assert_within("rstd", f64(o["rstd"]), r, 1.001 * U32 * r)
    # y: that, and two products
    slack = 3.01 * U32 * np.abs(y) + TINY
    if o["y"] is not None:
        assert_within("y", f64(o["y"]), y, slack + (0 if dt == F32 else HALF[dt] * np.abs(y) * (1 + 2.0 ** -10)))
    if o["y8"] is not None:
        check_rows8(o["y8"], o["scale"], y, slack)


def check_rows8(y8, scale, y, slack):
    """Codes and scales of values y known to within slack: a value's distance from
    its code is at most half a step, the scale that of the block's largest value."""
    T, d = y.shape
    codes, sb = codes_of(y8), scale.cpu().numpy().astype(np.int64)
    kb = CP(d) // 128
    assert not sb[:, kb:].any()
    assert not codes[:, d:].any()
    top = np.abs(ob.pad_to(y, CP(d))).reshape(T, kb, 128).max(axis=2)
    stop = ob.pad_to(slack, CP(d)).reshape(T, kb, 128).max(axis=2)
    e = sb[:, :kb] - 127
    assert np.all((e >= ob.block_exponent(np.maximum(top - stop, 0))) & (e <= ob.block_exponent(top + stop)))
    dec = ob.decode(codes, e)[:, :d]
    step = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * np.repeat(2.0 ** e.astype(float), 128, axis=1)[:, :d])
    assert_within("y8", dec, y, step * (1 + 2.0 ** -20) + 2 * slack)


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False], ids=["res", "plain"])
def test_forward(moe, T, d, dt, residual):
    announce(f"norm forward T={T} d={d} {dt} residual={residual}")
    x, gain = randn((T, d), 1.0, dt, 1), randn((d,), 1.0, dt, 2)
    res = randn((T, d), 3.0, dt, 3) if residual else None
    o = forward(moe, x, res, gain, 1e-5)
    torch.cuda.synchronize()
    check_forward(x, res, gain, 1e-5, o)
    if dt == F32:  # y is the unrounded value the 8-bit rows are made of: bit for bit the oracle's
        c, e = ob.encode(f64(o["y"]))
        assert np.array_equal(c, codes_of(o["y8"]))
        assert np.array_equal(ob.scale_bytes(e, d), o["scale"].cpu().numpy())
    # each output alone is the same as all together
    only = forward(moe, x, res, gain, 1e-5, y=True, q=False)
    assert torch.equal(only["y"], o["y"]) and torch.equal(only["rstd"], o["rstd"])
    only = forward(moe, x, res, gain, 1e-5, y=False, q=True)
    assert torch.equal(only["y8"].view(torch.uint8), o["y8"].view(torch.uint8))
    assert torch.equal(only["scale"], o["scale"])
    only = forward(moe, x, res, gain, 1e-5, y=False, q=False)
    assert torch.equal(only["rstd"], o["rstd"])


def test_extreme_rows(moe):
    """Zero rows (with and without eps), huge, tiny and non-finite values."""
    announce("norm extreme rows")
    d = 256
    x = randn((8, d), 1.0, F32, 5)
    x[0] = 0
    x[1] *= 1e15
    x[2] *= 1e-25
    x[3, 7] = float("inf")
    x[4, 200] = float("nan")
    x[5, 0] = 3e38
    x[5, 1:] = 0
    gain = torch.ones(d, device="cuda")
    o = forward(moe, x, None, gain, 1e-6)
    torch.cuda.synchronize()
    keep = [0, 1, 2, 5, 6, 7]
    sub = {k: (v[keep] if v is not None else None) for k, v in o.items()}
    check_forward(x[keep], None, gain, 1e-6, sub)
    y = f64(o["y"])
    assert not y[0].any() and not codes_of(o["y8"])[0].any() and (o["scale"].cpu().numpy()[0, :2] == 7).all()
    # an infinity: r = 0, its own value 0 * inf = NaN, the others 0; a NaN: the whole row
    assert np.isnan(y[3, 7]) and not y[3, :7].any() and np.isnan(y[4]).all()
    c = codes_of(o["y8"]) & 127
    assert c[3, 7] == 127 and (c[4] == 127).all()
    o = forward(moe, x[:1].contiguous(), None, gain, 0.0)  # 0 / 0
    assert torch.isnan(o["y"]).all() and torch.isinf(o["rstd"]).all()


@pytest.mark.parametrize("T,d", SHAPES + [(2100, 64), (1500, 576)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("with_dh", [True, False], ids=["dh", "nodh"])
def test_backward(moe, T, d, dt, with_dh):
    announce(f"norm backward T={T} d={d} {dt} dh={with_dh}")
    h, gain, dy = randn((T, d), 2.0, dt, 7), randn((d,), 1.0, dt, 8), randn((T, d), 1.0, dt, 9)
    dh = randn((T, d), 1.0, dt, 10) if with_dh else None
    p = moe.make_problem(T, d, 1, 1, 64, dt)
    rstd = forward(moe, h, None, gain, 1e-5, q=False)["rstd"]
    dx, dgain = torch.empty_like(h), torch.empty(d, dtype=F32, device="cuda")
    ws = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_NORM_BACKWARD), dtype=torch.uint8, device="cuda")
    moe.moex_add_rmsnorm_backward(p, h, gain, rstd, dy, dh, dx, dgain, ws)
    first = (dx.clone(), dgain.clone())
    moe.moex_add_rmsnorm_backward(p, h, gain, rstd, dy, dh, dx, dgain, ws)
    torch.cuda.synchronize()
    assert torch.equal(first[0], dx) and torch.equal(first[1], dgain)  # the same bits every time
    h64, g64, r, dy64 = f64(h), f64(gain), f64(rstd), f64(dy)
    dh64 = f64(dh) if with_dh else None
    rx, rg = ob.rmsnorm_backward(h64, g64, r, dy64, dh64)
    z, a = h64 * r[:, None], dy64 * g64
    # the mean of a z: at most 32 terms a thread, 6 + 16 more additions, a product each for a, z and 1/d
    n_mean = 32 + 6 + 16 + 4
    mean_abs = np.mean(np.abs(a * z), axis=1, keepdims=True)
    mag = r[:, None] * (np.abs(a) + np.abs(z) * np.abs(np.mean(a * z, axis=1, keepdims=True)))
    bound = 6 * U32 * mag + n_mean * U32 * r[:, None] * np.abs(z) * mean_abs
    if with_dh:
        bound = bound + U32 * (mag + np.abs(dh64))
    bound = bound + HALF[dt] * np.abs(rx) + TINY
    assert_within("dx", f64(dx), rx, bound)
    # dgain: no path adds more than its T terms and the tree's 16 + 16 + 4
    assert_within("dgain", f64(dgain), rg, (min(T, 64 + T // 64) + 40) * U32 * np.sum(np.abs(dy64 * z), axis=0) + TINY)


@pytest.mark.parametrize("T,d", [(1, 64), (5, 320), (777, 448), (3, 2112), (64, 7168)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_quantize_rows(moe, T, d, dt):
    announce(f"quantize rows T={T} d={d} {dt}")
    x = randn((T, d), 1.0, dt, 11)
    x[0, :64] = 0
    x *= torch.exp2(torch.randint(-60, 60, (T, 1), device="cuda")).to(dt)
    x[-1, -1] = float("nan")
    x[-1, 0] = float("inf")
    p = moe.make_problem(T, d, 1, 1, 64, dt)
    x8 = torch.full((T, CP(d)), 0x55, dtype=torch.uint8, device="cuda")
    xs = torch.full((T, SP(d)), 0x55, dtype=torch.uint8, device="cuda")
    moe.moex_quantize_rows(p, x, x8, xs)
    torch.cuda.synchronize()
    c, e = ob.encode(f64(x))
    got = x8.cpu().numpy()
    nan = (c & 127) == 127
    assert np.array_equal(nan, (got & 127) == 127) and nan.sum() >= (2 if T > 1 or d > 1 else 1)
    assert np.array_equal(c[~nan], got[~nan])
    assert np.array_equal(ob.scale_bytes(e, d), xs.cpu().numpy())


@pytest.mark.parametrize("T,d,dt", [(17000, 4096, BF), (8200, 4096, F32)], ids=["bf16", "f32"])
def test_large_arrays_pass_by_the_caches_with_the_same_bits(moe, T, d, dt):
    """Arrays of 128 MB and more take the streaming form; each half, below that, the plain one."""
    announce(f"norm large T={T} d={d} {dt}")
    x, res, gain = randn((T, d), 1.0, dt, 30), randn((T, d), 1.0, dt, 31), randn((d,), 1.0, dt, 32)
    o = forward(moe, x, res, gain, 1e-5)
    for half in (slice(0, T // 2), slice(T // 2, T)):
        part = forward(moe, x[half].contiguous(), res[half].contiguous(), gain, 1e-5)
        torch.cuda.synchronize()
        for key in ("h", "y", "scale", "rstd"):
            assert torch.equal(o[key][half], part[key]), key
        assert torch.equal(o["y8"][half].view(torch.uint8), part["y8"].view(torch.uint8))


def test_other_stream_and_inplace_refusal(moe):
    """Work goes to the stream given; an output over an input is refused before any of it."""
    announce("norm stream")
    T, d = 300, 512
    x, res, gain = randn((T, d), 1.0, BF, 33), randn((T, d), 1.0, BF, 34), randn((d,), 1.0, BF, 35)
    want = forward(moe, x, res, gain, 1e-5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = forward(moe, x, res, gain, 1e-5, stream=s)
    s.synchronize()
    assert torch.equal(want["y"], got["y"]) and torch.equal(want["h"], got["h"])
    p = moe.make_problem(T, d, 1, 1, 64, BF)
    keep = res.clone()
    with pytest.raises(moe.MoEError):
        moe.moex_add_rmsnorm(p, x, res, gain, 1e-5, res, want["y"], None, None, None)
    with pytest.raises(ValueError):
        moe.moex_add_rmsnorm(p, x[:, :256], res, gain, 1e-5, want["h"], want["y"], None, None, None)
    with pytest.raises(ValueError):
        moe.moex_add_rmsnorm(p, x.t().contiguous().t(), res, gain, 1e-5, want["h"], want["y"], None, None, None)
    with pytest.raises(TypeError):
        moe.moex_add_rmsnorm(p, x.float(), res, gain, 1e-5, want["h"], want["y"], None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(res, keep)


MANY = [(513, 64), (515, 576), (777, 1088), (514, 2112), (513, 4160), (515, 8256), (513, 16448)]


@pytest.mark.parametrize("T,d", MANY)
def test_forms_of_many_rows(moe, T, d):
    """More than 512 rows: several pieces per thread, the last of them not in every thread."""
    announce(f"norm many T={T} d={d}")
    for dt in (BF, F32) if d < 8000 else (BF,):
        x, res, gain = randn((T, d), 1.0, dt, 40), randn((T, d), 1.0, dt, 41), randn((d,), 1.0, dt, 42)
        o = forward(moe, x, res, gain, 1e-5)
        torch.cuda.synchronize()
        check_forward(x, res, gain, 1e-5, o)


@pytest.mark.parametrize("T,d", [(300, 7168), (1100, 2048)])
def test_codes_are_those_of_the_unrounded_result(moe, T, d):
    """bf16 rows and gains put many y next to ties of e4m3: no code may differ from
    the rounding of the float64 value (y is known to 2^-44, a tie that close does not occur)."""
    announce(f"norm codes T={T} d={d}")
    x, res, gain = randn((T, d), 1.0, BF, 50), randn((T, d), 1.0, BF, 51), randn((d,), 1.0, BF, 52)
    o = forward(moe, x, res, gain, 1e-5)
    torch.cuda.synchronize()
    y, _ = ob.rmsnorm(f64(o["h"]), f64(gain), float(np.float32(1e-5)))
    want, e = ob.encode(ob.pad_to(y, CP(d)))
    got = codes_of(o["y8"])
    assert np.array_equal(o["scale"].cpu().numpy()[:, : CP(d) // 128], e + 127)
    assert np.array_equal(got, want)
    # infinite and zero gains, rows of zeros: the correction adds nothing of its own
    gain[:3] = torch.tensor([float("inf"), float("-inf"), 0.0])
    x[0].zero_()
    o = forward(moe, x, None, gain, 1e-5)
    torch.cuda.synchronize()
    f = o["y"].float()
    assert torch.isnan(f[0, :2]).all() and not f[0, 2:].any()
    r = f[1:][x[1:, 0] != 0]
    assert torch.isinf(r[:, 0]).all() and torch.isfinite(r[:, 2:]).all()
    assert (o["scale"][1:, 0][x[1:, 0] != 0] == 247).all()


@pytest.mark.parametrize("T,d", [(1100, 320), (1090, 1088), (1030, 2112), (1026, 4160), (1025, 8192)])
def test_backward_of_many_rows(moe, T, d):
    """More than 1024 rows: dgain by partial sums and a second launch."""
    for dt in (BF, F32) if d < 4000 else (BF,):
        test_backward(moe, T, d, dt, True)


def test_rows_whose_root_overflows_keep_their_infinities(moe):
    """eps 0 and rows of 1e-42: r is past float32, y infinite, its block at the largest scale."""
    announce("norm infinite r")
    x = torch.full((3, 256), 1e-42, dtype=F32, device="cuda")
    x[1] = 1.0
    o = forward(moe, x, None, torch.ones(256, dtype=F32, device="cuda"), 0.0)
    torch.cuda.synchronize()
    for t in (0, 2):
        assert torch.isinf(o["rstd"][t]) and torch.isinf(o["y"][t]).all() and (o["scale"][t, :2] == 247).all()
        assert torch.isnan(o["y8"][t].float()).all()
    assert (o["y"][1] == 1).all() and (o["scale"][1, :2] == 119).all()
