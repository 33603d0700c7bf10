"""Plain float64 forms of what trains the layer's surroundings (NumPy; TEST
INFRASTRUCTURE ONLY, imported by tests, never by the product path).

Each function is the definition written out: a sort by (expert, selection), sums
over rows, the derivatives of the activations, the optimizer's formulas, and a
stochastic rounding that looks up the two neighbouring codes.
"""

from __future__ import annotations

import math
from typing import Dict, Optional

import numpy as np

from .block_ops import E4M3


# ---- rows sorted by expert and back

def dispatch_index(idx: np.ndarray, E: int) -> Dict[str, np.ndarray]:
    """counts, offsets, perm (rows of live selections only), inv of topk_idx [T, k]; entries outside [0, E) are dropped."""
    T, k = idx.shape
    flat = idx.reshape(-1).astype(np.int64)
    live = np.nonzero((flat >= 0) & (flat < E))[0]
    order = live[np.argsort(flat[live], kind="stable")]
    inv = np.full(T * k, -1, np.int64)
    inv[order] = np.arange(order.size)
    counts = np.bincount(flat[live], minlength=E)
    return {"counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]), "perm": order // k, "inv": inv,
            "order": order}


def to_rows(src: np.ndarray, index, weight: Optional[np.ndarray]) -> np.ndarray:
    """Rows [live, d]: weight[t, j] src[t] of each row's selection."""
    rows = src[index["perm"]]
    return rows if weight is None else rows * weight.reshape(-1)[index["order"]][:, None]


def from_rows(rows: np.ndarray, index, weight: Optional[np.ndarray], add: Optional[np.ndarray], T: int) -> np.ndarray:
    """add[t] + sum over the selections of token t of weight times their row."""
    out = np.zeros((T, rows.shape[1])) if add is None else add.copy()
    live = rows[:index["perm"].size]
    if weight is not None:
        live = live * weight.reshape(-1)[index["order"]][:, None]
    np.add.at(out, index["perm"], live)
    return out


def dots(rows: np.ndarray, tokens: np.ndarray, index, k: int) -> np.ndarray:
    """<tokens[t], row of (t, j)> [T, k], 0 where dropped."""
    out = np.zeros(tokens.shape[0] * k)
    n = index["perm"].size
    out[index["order"]] = np.sum(rows[:n] * tokens[index["perm"]], axis=1)
    return out.reshape(-1, k)


def softmax_rows(logits: np.ndarray) -> np.ndarray:
    """Row softmax; a row of -infinity alone has probability 0 everywhere."""
    top = np.max(logits, axis=1, keepdims=True)
    e = np.exp(logits - np.where(np.isfinite(top), top, 0.0))
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def gate_backward(logits: np.ndarray, idx: np.ndarray, dgate: np.ndarray, add: Optional[np.ndarray]) -> np.ndarray:
    T, E = logits.shape
    q = softmax_rows(logits)
    dp = np.zeros((T, E))
    for t in range(T):
        for j in range(idx.shape[1]):
            if 0 <= idx[t, j] < E:
                dp[t, idx[t, j]] += dgate[t, j]
    out = q * (dp - np.sum(q * dp, axis=1, keepdims=True))
    return out if add is None else out + add


# ---- a dense projection

def act(u: np.ndarray, name: str) -> np.ndarray:
    if name == "gelu":
        return 0.5 * u * (1 + np.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
    if name == "silu":
        return u / (1 + np.exp(-u))
    return np.maximum(u, 0) if name == "relu" else u


def act_slope(u: np.ndarray, name: str) -> np.ndarray:
    if name == "gelu":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (u + 0.044715 * u ** 3))
        return 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * c * (1 + 3 * 0.044715 * u * u)
    if name == "silu":
        s = 1 / (1 + np.exp(-u))
        return s + u * s * (1 - s)
    return (u > 0).astype(np.float64) if name == "relu" else np.ones_like(u)


# ---- the optimizer's step

def e5m2_values() -> np.ndarray:
    """Value of every non-negative e5m2 code below infinity (5 exponent bits of bias 15, 2 mantissa bits)."""
    return np.array([(c & 3) / 4 * 2.0 ** -14 if c < 4 else (1 + (c & 3) / 4) * 2.0 ** ((c >> 2) - 15) for c in range(124)])


E4M3_POS, E5M2_POS = E4M3[:127], e5m2_values()


def mix(x: int) -> int:
    x &= 0xFFFFFFFF
    x ^= x >> 16
    x = x * 0x7FEB352D & 0xFFFFFFFF
    x ^= x >> 15
    x = x * 0x846CA68B & 0xFFFFFFFF
    return x ^ (x >> 16)


def draws(n: int, seed: int, t: int, tensor: int, first: int = 0) -> np.ndarray:
    """The 32-bit random number of elements first .. first + n - 1 (Python integers; small n)."""
    key = mix(seed + mix(0x9E3779B9 * t + tensor))
    return np.array([mix(((i & 0xFFFFFFFF) + key & 0xFFFFFFFF) ^ (0x9E3779B9 * (i >> 32) & 0xFFFFFFFF))
                     for i in range(first, first + n)], dtype=np.int64)


def block_exponent(amax: np.ndarray, top: float) -> np.ndarray:
    """Smallest e in [-120, 120] with amax <= top 2^e."""
    e = np.full(amax.shape, -120, np.int64)
    for v in range(-120, 120):
        e = np.where(amax > top * 2.0 ** v, v + 1, e)
    return e


def round_stochastic(x: np.ndarray, r: np.ndarray, table: np.ndarray, keep: bool):
    """(codes, exponents) of a tensor's values with 16-bit random numbers r. With lo the largest code's value
    not above |x| and s the distance to the next, |x| becomes the next one when |x| - lo + s r / 65536 >= s."""
    n = x.size
    pad = -n % 128
    a = np.abs(np.pad(x, (0, pad))).reshape(-1, 128)
    e = block_exponent(np.max(np.where(np.isnan(a), 0.0, a), axis=1), table[-1])  # NaN is left out
    v = np.ldexp(a, -e[:, None].astype(np.int32)).reshape(-1)[:n]
    bad = ~(v <= table[-1])
    v = np.where(bad, 0.0, v)
    lo = np.searchsorted(table, v, side="right") - 1
    s = table[np.minimum(lo + 1, table.size - 1)] - table[lo]
    s = np.where(s == 0, 1.0, s)
    up = np.floor((v - table[lo]) / s * 65536) + r >= 65536
    code = lo + (up & (lo + 1 < table.size))
    if keep:
        code = np.where((code == 0) & (v > 0), 1, code)
    code = np.where(bad, 0x7F, code) + (0 if keep else 128 * np.signbit(x))
    return code.astype(np.uint8), e


def decode(codes: np.ndarray, e: np.ndarray, table: np.ndarray) -> np.ndarray:
    full = np.full(128, np.nan)
    full[:table.size] = table
    v = full[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    return v * np.exp2(np.repeat(e, 128)[:codes.size].astype(np.float64))


def adamw(param: np.ndarray, grad: np.ndarray, m: np.ndarray, v: np.ndarray, t: int, lr: float, beta1: float, beta2: float,
          eps: float, decay: float):
    """(param, m, v) after step t, all float64."""
    m = beta1 * m + (1 - beta1) * grad
    v = beta2 * v + (1 - beta2) * grad * grad
    step = m / -math.expm1(t * math.log(beta1) if beta1 else -math.inf)
    step = step / (np.sqrt(v / -math.expm1(t * math.log(beta2) if beta2 else -math.inf)) + eps)
    return param - lr * (step + decay * param), m, v
