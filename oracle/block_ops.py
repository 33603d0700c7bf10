"""Plain float64 forms of the operators around the layer (NumPy; TEST
INFRASTRUCTURE ONLY, imported by tests, never by the product path).

Each function is the definition written out on exact input values: the e4m3
code table is built from the format's fields, rounding picks the nearest code
(ties to the even one), nothing is blocked or fused.
"""

from __future__ import annotations

import math
from typing import Dict, Optional, Tuple

import numpy as np


def e4m3_values() -> np.ndarray:
    """Value of every e4m3 code (4 exponent bits of bias 7, 3 mantissa bits, no infinity)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if s else v
    return out


E4M3 = e4m3_values()
_POS = E4M3[:127]  # 0 .. 448, increasing


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Codes of float64 values: nearest, ties to even; past 464 and non-finite: NaN codes."""
    a = np.abs(v)
    fin = np.isfinite(a) & (a <= 464.0)
    aa = np.where(fin, a, 0.0)
    hi = np.minimum(np.searchsorted(_POS, aa, side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = aa - _POS[lo], _POS[hi] - aa
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(aa >= 448.0, 126, code)
    code = np.where(fin, code, 127)
    return (code + 128 * np.signbit(v)).astype(np.uint8)


def block_exponent(amax: np.ndarray) -> np.ndarray:
    """Smallest e in [-120, 120] with amax <= 448 2^e."""
    m, q = np.frexp(np.where(np.isfinite(amax), amax, 0.0))  # amax = m 2^q, m in [0.5, 1); 448 = 0.875 2^9
    e = np.clip(q - 9 + (m > 0.875), -120, 120)
    e = np.where(amax == 0, -120, e)
    return np.where(np.isinf(amax), 120, e).astype(np.int64)


def pad_to(v: np.ndarray, n: int) -> np.ndarray:
    w = [(0, 0)] * (v.ndim - 1) + [(0, n - v.shape[-1])]
    return np.pad(v, w)


def code_pitch(K: int) -> int:
    return -(-K // 128) * 128


def scale_pitch(K: int) -> int:
    return -(-K // 2048) * 16


def encode(v: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(codes [..., Kp], exponents [..., Kp / 128]) of rows of values."""
    b = pad_to(v, code_pitch(v.shape[-1]))
    b = b.reshape(*b.shape[:-1], -1, 128)
    e = block_exponent(np.nanmax(np.where(np.isnan(b), 0.0, np.abs(b)), axis=-1))
    with np.errstate(invalid="ignore", over="ignore"):
        codes = round_e4m3(np.ldexp(b, -e[..., None].astype(np.int32)))
    return codes.reshape(*v.shape[:-1], -1), e


def decode(codes: np.ndarray, e: np.ndarray) -> np.ndarray:
    b = E4M3[codes].reshape(*codes.shape[:-1], -1, 128)
    return np.ldexp(b, e[..., None].astype(np.int32)).reshape(codes.shape)


def scale_bytes(e: np.ndarray, K: int) -> np.ndarray:
    return pad_to((e + 127).astype(np.uint8), scale_pitch(K))


def weight_layout(w: np.ndarray) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """Expert weights [E, K, N]: (codes, scale bytes) in the matrix-core layout, and the decoded weights."""
    E, K, N = w.shape
    codes, e = encode(np.swapaxes(w, 1, 2))  # [E, N, Kp], [E, N, KB]
    KB = e.shape[-1]
    q = np.empty((E, N // 32, KB, 4, 2, 32, 16), np.uint8)
    for h in range(2):
        for qq in range(4):
            k0 = 32 * qq + 16 * h
            src = codes.reshape(E, N // 32, 32, KB, 128)[..., k0:k0 + 16]
            q[:, :, :, qq, h] = np.swapaxes(src, 2, 3)
    s = np.swapaxes((e + 127).astype(np.uint8).reshape(E, N // 32, 32, KB), 2, 3)
    return q, np.ascontiguousarray(s), np.swapaxes(decode(codes, e), 1, 2)


def rmsnorm(h: np.ndarray, gain: np.ndarray, eps: float) -> Tuple[np.ndarray, np.ndarray]:
    """(y, rstd) of rows h."""
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * r[:, None] * gain, r


def rmsnorm_backward(h, gain, r, dy, dh=None) -> Tuple[np.ndarray, np.ndarray]:
    """(dx, dgain)."""
    z, a = h * r[:, None], dy * gain
    dx = r[:, None] * (a - z * np.mean(a * z, axis=1, keepdims=True))
    return (dx if dh is None else dx + dh), np.sum(dy * z, axis=0)


def softmax_rows(logits: np.ndarray) -> np.ndarray:
    """Softmax of rows; a row of -infinity alone has no probability anywhere."""
    m = logits.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(m == -np.inf, 0.0, np.exp(logits - m))
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s != 0)


def balance_loss(logits, idx, mask, coef) -> Dict[str, np.ndarray]:
    T, E = logits.shape
    k = idx.shape[1]
    valid = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    n = int(valid.sum())
    sel = idx[valid].reshape(-1)
    counts = np.bincount(sel[(sel >= 0) & (sel < E)], minlength=E)
    dl, P = np.zeros((T, E)), np.zeros(E)
    if n == 0:
        return {"loss": 0.0, "counts": counts, "mean_prob": P, "dlogits": dl, "p": dl}
    p = np.zeros((T, E))
    p[valid] = softmax_rows(logits[valid])
    P = p.sum(axis=0) / n
    f = counts / (n * k)
    dl = coef * E / n * p * (f - (p @ f)[:, None])
    return {"loss": coef * E * float(f @ P), "counts": counts, "mean_prob": P, "dlogits": dl, "p": p}


def gelu_tanh(u: np.ndarray) -> np.ndarray:
    return 0.5 * u * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (u + 0.044715 * u ** 3)))


def grouped_ffn_fp8(x: np.ndarray, offsets, w1: np.ndarray, w2: np.ndarray, hidden: Optional[dict] = None):
    """y_perm of decoded rows x (already permuted) and decoded weights [E, Kp, N];
    rows outside every group are NaN. hidden: filled with U per expert."""
    R, d = x.shape[0], w2.shape[2]
    y = np.full((R, d), np.nan)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        u = x[lo:hi] @ w1[e]
        if hidden is not None:
            hidden[e] = u
        codes, ex = encode(gelu_tanh(u))
        y[lo:hi] = decode(codes, ex) @ w2[e]
    return y
