"""Shared helpers of the tests of the operators around the layer (not collected as tests)."""

from __future__ import annotations

import numpy as np
import torch

from gpu_helpers import U32, f64
from oracle import block_ops as ob

# relative half step of a rounding to each type
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 1e-37  # below every normal float32: absolute slack where results underflow


def gen(seed: int) -> torch.Generator:
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, std, dtype, seed):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(dtype)


def codes_of(t: torch.Tensor) -> np.ndarray:
    return t.view(torch.uint8).cpu().numpy()


def quantized(moe, x: torch.Tensor):
    """(codes, scale bytes, decoded float64 values [T, Kp]) of rows by the oracle, on the GPU and host."""
    v = f64(x)
    c, e = ob.encode(v)
    s = ob.scale_bytes(e, v.shape[1])
    return torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), ob.decode(c, e)


def ffn_bound(x, offsets, w1, w2, de):
    """(y, bound) of the 8-bit expert FFN for decoded rows x (permuted) and weights.

    The sums of one matrix instruction over 64 positions are off by at most
    2^-11 of its largest product (products are aligned to it before they are
    added; 2^-11.8 is the most seen over random codes of the full range), and
    each of the K / 64 additions to the float32 accumulator, and of the up to
    16 partial sums, by 2^-24 of the sum of magnitudes. GELU has a slope of at
    most 1.13 and adds 2^-20 of its argument's size for its hardware exponential
    and reciprocal (each within 2^-22). A hidden value's code differs where the
    value, within that slack, reaches another code or another block scale; it
    then differs by what the oracle's encoding of the shifted values differs.
    """
    R, d = x.shape[0], w2.shape[2]
    y, bound = np.full((R, d), np.nan), np.zeros((R, d))

    def product(a, b):
        K, out, err = a.shape[1], a @ b, 0.0
        aa, bb = np.abs(a), np.abs(b)
        for k in range(0, K, 64):
            err = err + 2.0 ** -11 * np.max(aa[:, k:k + 64, None] * bb[None, k:k + 64], axis=1)
        return out, err + (K / 64 + 16) * U32 * (aa @ bb)

    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        u, du = product(x[lo:hi], w1[e])
        h = ob.gelu_tanh(u)
        dh = 1.13 * du + 2.0 ** -20 * np.abs(u)
        ref = ob.decode(*ob.encode(h))
        far = np.zeros_like(ref)
        for sh in (h - dh, h + dh):  # every element moved down, then up: codes and scales move with them
            far = np.maximum(far, np.abs(ob.decode(*ob.encode(sh)) - ref))
        # the largest value of a block moving alone can change the scale under unmoved values
        grow = h + np.where(h >= 0, 1.0, -1.0) * dh
        shrink = np.where(h >= 0, 1.0, -1.0) * np.maximum(np.abs(h) - dh, 0.0)
        for sh in (grow, shrink):
            far = np.maximum(far, np.abs(ob.decode(*ob.encode(sh)) - ref))
            ex = ob.block_exponent(np.max(np.abs(ob.pad_to(sh, ref.shape[1])).reshape(len(sh), -1, 128), axis=2))
            b = ob.pad_to(h, ref.shape[1]).reshape(len(h), -1, 128)
            alt = ob.E4M3[ob.round_e4m3(np.clip(np.ldexp(b, -ex[..., None].astype(np.int32)), -448, 448))]
            far = np.maximum(far, np.abs(np.ldexp(alt, ex[..., None].astype(np.int32)).reshape(ref.shape) - ref))
        out, dy = product(ref, w2[e])
        y[lo:hi] = out
        bound[lo:hi] = dy + far @ np.abs(w2[e])
    return y, bound + HALF[torch.bfloat16] * np.abs(np.nan_to_num(y))


def assert_within(name, got, ref, bound):
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(got - ref) - bound), got.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside the bound, worst at {i}: got {got[i]!r}, "
                             f"expected {ref[i]!r} within {np.broadcast_to(bound, got.shape)[i]!r}")
