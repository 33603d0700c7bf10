"""Measured cases of the operators that train the sparse mixture-of-experts layer's surroundings.

Three operators, each with a plain form (elementary torch operations in
float32) and the library's own calls:

  tokens    selections sorted by expert and the rows brought there and back,
            with the gates applied on either way; in training also the
            gradients of both ways and of the router's logits
  linear    y = residual + act(x W + bias) for a dense projection beside the
            experts; in training also the gradients of x, W and bias
  adamw     one AdamW step over a list of tensors, with the global norm of the
            gradients and clipping, and moments in 32 or in 8 bits

Moments in 8 bits: 128 consecutive values of a tensor share a scale 2^e, e the
smallest integer with max <= top * 2^e (kept in [-120, 120], held as the byte
e + 127); the first moment is held as e4m3 codes (top 448), the second as e5m2
codes (top 57344). Codes are rounded stochastically: with s the spacing of
codes at |x| and r the element's 16-bit random number, |x| becomes
s floor(|x| / s + r / 65536); a second moment that is not 0 is never rounded to
0. Element i of tensor j at step t draws, in 32-bit arithmetic,
  mix((lo32(i) + mix(seed + mix(0x9E3779B9 t + j))) ^ (0x9E3779B9 hi32(i)))
whose low half is the first moment's number and whose high half the second's.
"""

import math
import random

import torch

own = False

LR, BETA1, BETA2, ADAM_EPS, DECAY, SEED = 3e-4, 0.9, 0.999, 1e-8, 0.1, 20
STEPS = 1000  # taken before the measured one


# ---------------------------------------------------------------- the cases

def _tokens(name, T, d, E, k, dtype, early, train, drop):
    return {"name": name, "op": "tokens", "T": T, "d": d, "E": E, "k": k, "dtype": dtype, "early": early, "train": train,
            "drop": drop}


def _linear(name, T, K, N, act, bias, residual, train):
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "act": act, "bias": bias, "residual": residual,
            "train": train}


def _layer(name, d, E, de, bits, clip):
    return {"name": name, "op": "adamw", "kind": "layer", "d": d, "E": E, "de": de, "bits": bits, "clip": clip}


def _ragged(name, count, largest, sizes, bits, clip):
    return {"name": name, "op": "adamw", "kind": "ragged", "count": count, "largest": largest, "sizes": sizes,
            "bits": bits, "clip": clip}


def listed():
    return [
        # a decode batch of 32 through a fine-grained layer: latency counts
        _tokens("tokens_decode_32x2048", 32, 2048, 64, 8, "bf16", False, False, 0.0),
        # ragged float32 rows with dropped selections, gates applied on the way to the experts, both directions
        _tokens("tokens_train_777x320_f32", 777, 320, 12, 3, "f32", True, True, 0.1),
        # a training step of the fine-grained layer
        _tokens("tokens_train_8192x2048", 8192, 2048, 64, 8, "bf16", False, True, 0.0),
        # a prefill of the large sparse layer
        _tokens("tokens_16384x7168", 16384, 7168, 256, 8, "bf16", False, False, 0.0),
        # one token through a dense expert's first product
        _linear("linear_decode_1x2048x8192", 1, 2048, 8192, "gelu", True, False, False),
        # a decode batch of 32 through its second, added to the routed experts' output
        _linear("linear_decode_32x8192x2048", 32, 8192, 2048, "none", True, True, False),
        # an odd number of rows of odd multiples of 64, both directions
        _linear("linear_train_777x320x448", 777, 320, 448, "silu", True, True, True),
        # a training step's first product of a dense expert as wide as the coarse ones
        _linear("linear_train_8192x2048x8192", 8192, 2048, 8192, "gelu", True, False, True),
        # the tiny layer's parameters: launch latency
        _layer("adamw_tiny", 128, 8, 256, 32, True),
        # sixteen of the fine-grained experts, moments in 32 bits
        _layer("adamw_16x2048x1024", 2048, 16, 1024, 32, True),
        # the same with moments in 8 bits
        _layer("adamw_16x2048x1024_8bit", 2048, 16, 1024, 8, True),
        # many tensors of odd sizes
        _ragged("adamw_48_tensors_8bit", 48, 1 << 20, 1, 8, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("tokens", "linear", "adamw"))
    if op == "tokens":
        E = _log_int(rng, 1, 256)
        k, d, train = rng.randint(1, min(E, 8)), 64 * _log_int(rng, 1, 112), rng.random() < 0.5
        T = min(_log_int(rng, 1, 16384), (1 << 27 if train else 1 << 29) // (d * k))
        return {"op": op, "T": T, "d": d, "E": E, "k": k, "dtype": rng.choice(("bf16", "bf16", "f32")),
                "early": rng.random() < 0.4, "train": train, "drop": rng.choice((0.0, 0.0, 0.1, 0.6))}
    if op == "linear":
        K, N, train = 64 * _log_int(rng, 1, 128), 64 * _log_int(rng, 1, 128), rng.random() < 0.5
        return {"op": op, "T": min(_log_int(rng, 1, 8192), max(1, (1 << 37) // (K * N))), "K": K, "N": N,
                "act": rng.choice(("none", "gelu", "silu", "relu")), "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.5, "train": train}
    bits, clip = rng.choice((8, 32)), rng.random() < 0.6
    if rng.random() < 0.4:
        d, de = 64 * _log_int(rng, 1, 32), 64 * _log_int(rng, 1, 32)
        return {"op": op, "kind": "layer", "d": d, "E": min(_log_int(rng, 1, 32), (1 << 25) // (d * de)), "de": de,
                "bits": bits, "clip": clip}
    return {"op": op, "kind": "ragged", "count": _log_int(rng, 1, 96), "largest": _log_int(rng, 1, 1 << 20),
            "sizes": rng.randint(1, 1 << 20), "bits": bits, "clip": clip}


def _sizes(case):
    """(values, type, bits of the moments) of each tensor of a list."""
    if case["kind"] == "layer":
        d, E, de = case["d"], case["E"], case["de"]
        shapes = [(E * d * de, "bf16"), (E * d * de, "bf16"), (d * E, "bf16"), (d, "bf16"), (E, "f32")]
    else:
        rng = random.Random(case["sizes"])
        shapes = [(_log_int(rng, 1, case["largest"]), "f32" if rng.random() < 0.25 else "bf16")
                  for _ in range(case["count"])]
    # moments of small tensors are not worth 8 bits
    return [(n, dt, case["bits"] if n >= 4096 else 32) for n, dt in shapes]


def work(case):
    if case["op"] == "adamw":
        total = 0
        for n, dt, bits in _sizes(case):
            # gradient in; master (bf16 rows: beside the parameter) in and out, both moments in and out
            total += n * ((2 + 8 + 2) if dt == "bf16" else (4 + 8)) + n * (4 if bits == 8 else 16)
            total += 2 * 2 * (n // 128) if bits == 8 else 0
        return {"bytes": total, "flops": 20 * sum(n for n, _, _ in _sizes(case))}
    T = case["T"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        io = T * K + K * N + T * N * (2 if case["residual"] else 1)
        if not case["train"]:
            return {"bytes": 2 * io, "flops": 2 * T * K * N}
        # u out and in; dy in, dx and dW out
        return {"bytes": 2 * (io + 3 * T * N + T * K + K * N), "flops": 6 * T * K * N}
    d, k, es = case["d"], case["k"], 2 if case["dtype"] == "bf16" else 4
    rows = T * k * d * es * (1.0 - case["drop"])
    # x and the residual in, y out, every row written once and read once
    total = 3 * T * d * es + 2 * rows + 20 * T * k
    if case["train"]:
        # dy in, rows of its gradient out; rows of x's gradient in, the other way's gradient in and dx out;
        # the rows that the gates' gradient needs once more are read above
        total += 3 * T * d * es + 2 * rows + 8 * T * case["E"]
    return {"bytes": int(total), "flops": int((10 if case["train"] else 3) * T * k * d)}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _up(n, m):
    return (n + m - 1) // m * m


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _prepare_tokens(case, g):
    T, d, E, k, dt = case["T"], case["d"], case["E"], case["k"], _DT[case["dtype"]]
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((E,), generator=g, device="cuda")
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    gate = torch.softmax(logits, dim=1).gather(1, order).contiguous()
    gone = torch.rand((T, k), generator=g, device="cuda") < case["drop"]
    s = {"logits": logits.contiguous(), "gate": gate,
         "idx": torch.where(gone, torch.full_like(order, -1), order).to(torch.int32).contiguous(),
         "x": _normal(g, (T, d), 1.0, dt), "y_perm": _normal(g, (T * k, d), 1.0, dt),
         "residual": _normal(g, (T, d), 2.0, dt)}
    if case["train"]:
        s["dy"] = _normal(g, (T, d), 1.0, dt)
        s["dx_perm"] = _normal(g, (T * k, d), 1.0, dt)
        s["dh"] = _normal(g, (T, d), 1.0, dt)
    return s


def _prepare_linear(case, g):
    T, K, N = case["T"], case["K"], case["N"]
    s = {"x": _normal(g, (T, K), 1.0, torch.bfloat16), "W": _normal(g, (K, N), K ** -0.5, torch.bfloat16),
         "bias": _normal(g, (N,), 0.3, torch.bfloat16) if case["bias"] else None,
         "residual": _normal(g, (T, N), 1.0, torch.bfloat16) if case["residual"] else None}
    if case["train"]:
        s["dy"] = _normal(g, (T, N), 1.0, torch.bfloat16)
    return s


def _pow2(e):
    """2^e in 64 bits; torch.ldexp goes by a power in 32 bits that is not exact."""
    return torch.exp2(e.double())


def _nearest_codes(x, top, dtype):
    """Rows of 128 float32 values as codes of `dtype` and scale bytes, rounded to nearest."""
    m = x.abs().amax(dim=1)
    e = torch.ceil(torch.log2(m.double() / top).clamp(-120, 120)).to(torch.int32)
    e = torch.where(m > 0, e, torch.full_like(e, -120))
    return (x * _pow2(-e)[:, None]).clamp(-top, top).to(dtype), (e + 127).to(torch.uint8)


def _prepare_adamw(case, g):
    """Parameters, gradients and moments in one buffer of each kind, as views whose addresses are multiples of 256 bytes."""
    sizes = _sizes(case)
    n16 = sum(_up(n, 128) for n, dt, _ in sizes if dt == "bf16")
    n32 = sum(_up(n, 128) for n, dt, _ in sizes if dt == "f32")
    m32 = sum(_up(n, 128) for n, _, b in sizes if b == 32)
    m8 = sum(_up(n, 128) for n, _, b in sizes if b == 8)
    s8 = sum(_up(_up(n, 128) // 128, 256) for n, _, b in sizes if b == 8)
    master = torch.randn((n16,), generator=g, device="cuda") * 0.03
    flat = {"bf16": master.to(torch.bfloat16), "f32": torch.randn((n32,), generator=g, device="cuda") * 0.03, "master": master}

    def grads(n):  # rows of 128 of different size, as rows of different experts have
        size = torch.exp2(3.0 * torch.randn((n // 128, 1), generator=g, device="cuda") - 10.0)
        return size, (torch.randn((n // 128, 128), generator=g, device="cuda") * size)

    def moments(size):
        shape = (size.shape[0], 128)
        m = torch.randn(shape, generator=g, device="cuda") * size * 0.3
        v = (torch.randn(shape, generator=g, device="cuda").square() * 0.3 + 0.5) * size.square()
        return m, v

    size16, g16 = grads(n16)
    size32, g32 = grads(n32)
    flat["g_bf16"], flat["g_f32"] = g16.reshape(-1).to(torch.bfloat16), g32.reshape(-1)
    mv = {"bf16": moments(size16), "f32": moments(size32)}
    flat["m32"], flat["v32"] = torch.zeros((m32,), device="cuda"), torch.zeros((m32,), device="cuda")
    flat["m8"] = torch.zeros((m8,), device="cuda").to(torch.float8_e4m3fn)
    flat["v8"] = torch.zeros((m8,), device="cuda").to(torch.float8_e5m2)
    flat["ms"], flat["vs"] = (torch.full((s8,), 7, dtype=torch.uint8, device="cuda") for _ in range(2))
    at = {"bf16": 0, "f32": 0, 32: 0, 8: 0, "s": 0}
    s = {"flat": flat, "param": [], "grad": [], "master": [], "m": [], "v": [], "m_scale": [], "v_scale": []}
    for n, dt, bits in sizes:
        a, b, N = at[dt], at[bits], _up(n, 128)
        at[dt] += N
        at[bits] += N
        s["param"].append(flat[dt][a:a + n])
        s["grad"].append(flat["g_" + dt][a:a + n])
        s["master"].append(flat["master"][a:a + n] if dt == "bf16" else None)
        m, v = (t[a // 128:(a + N) // 128] for t in mv[dt])
        if bits == 32:
            s["m"].append(flat["m32"][b:b + n])
            s["v"].append(flat["v32"][b:b + n])
            s["m"][-1].copy_(m.reshape(-1)[:n])
            s["v"][-1].copy_(v.reshape(-1)[:n])
            s["m_scale"].append(None)
            s["v_scale"].append(None)
            continue
        inside = (torch.arange(N, device="cuda") < n).view(-1, 128)
        c = at["s"]
        at["s"] += _up(N // 128, 256)
        for key, val, top, ct in (("m", m, 448.0, torch.float8_e4m3fn), ("v", v, 57344.0, torch.float8_e5m2)):
            codes, scale = _nearest_codes(val * inside, top, ct)
            s[key].append(flat[key + "8"][b:b + n])
            s[key + "_scale"].append(flat[key + "s"][c:c + N // 128])
            s[key][-1].copy_(codes.reshape(-1)[:n])
            s[key + "_scale"][-1].copy_(scale)
    s["counter"] = torch.tensor([STEPS, 0], dtype=torch.int32, device="cuda")
    # half of the norm that these gradients have: the step is clipped
    norm = torch.sqrt(sum(t.double().square().sum() for t in s["grad"]))
    s["max_norm"] = float(norm) / 2 if case["clip"] else None
    return s


def prepare(case, seed):
    g = _gen(seed)
    s = {"tokens": _prepare_tokens, "linear": _prepare_linear, "adamw": _prepare_adamw}[case["op"]](case, g)
    s["case"] = case
    return s


# ---------------------------------------------------------------- plain forms

def _plain_tokens(s):
    case, x, idx = s["case"], s["x"], s["idx"].long()
    T, E, k, dt = case["T"], case["E"], case["k"], x.dtype
    R, dev = T * k, x.device
    flat = idx.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    r = torch.arange(R, device=dev)
    live = r < offsets[E]
    inv = torch.empty_like(order)
    inv[order] = torch.where(live, r, torch.full_like(r, -1))
    kept = (inv >= 0)[:, None]
    gate = s["gate"].reshape(-1, 1)
    w_in, w_out = (gate, None) if case["early"] else (None, gate)

    def to_rows(t, w):  # row r: its token's row of t, times its weight
        rows = t.float()[order // k]
        rows = rows if w is None else rows * w[order]
        return torch.where(live[:, None], rows, torch.zeros_like(rows)).to(dt)

    def from_rows(rows, w, add):
        v = torch.where(kept, rows.float()[inv.clamp(min=0)], torch.zeros((), device=dev))
        v = v if w is None else v * w
        return (v.view(T, k, -1).sum(dim=1) + add.float()).to(dt)

    def dots(rows, t):  # of each selection's row with its token's row
        v = torch.where(kept, rows.float()[inv.clamp(min=0)], torch.zeros((), device=dev))
        return (v.view(T, k, -1) * t.float()[:, None, :]).sum(dim=2)

    out = {"counts": counts.to(torch.int32), "offsets": offsets.to(torch.int32), "inv": inv.to(torch.int32),
           "perm": torch.where(live, order // k, torch.zeros_like(order)).to(torch.int32), "x_perm": to_rows(x, w_in),
           "y": from_rows(s["y_perm"], w_out, s["residual"])}
    if not case["train"]:
        return out
    out["dy_perm"] = to_rows(s["dy"], w_out)
    out["dx"] = from_rows(s["dx_perm"], w_in, s["dh"])
    out["dgate"] = dots(s["dx_perm"], x) if case["early"] else dots(s["y_perm"], s["dy"])
    e = torch.exp(s["logits"] - s["logits"].amax(dim=1, keepdim=True))
    p = e / e.sum(dim=1, keepdim=True)
    key = key.view(T, k)
    dp = torch.zeros((T, E + 1), device=dev)
    dp = dp.scatter_add(1, key, out["dgate"])[:, :E]
    out["dlogits"] = p * (dp - (p * dp).sum(dim=1, keepdim=True))
    return out


def _act(u, act):
    """(act(u), its derivative)."""
    if act == "none":
        return u, torch.ones_like(u)
    if act == "relu":
        return torch.where(u > 0, u, torch.zeros_like(u)), (u > 0).to(u.dtype)
    if act == "silu":
        h = 1.0 / (1.0 + torch.exp(-u))
        return u * h, h * (1.0 + u * (1.0 - h))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (u + 0.044715 * u * u * u))
    return 0.5 * u * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * u * (1.0 - t * t) * c * (1.0 + 0.134145 * u * u)


def _plain_linear(s):
    case, x, W = s["case"], s["x"].float(), s["W"].float()
    u = x @ W
    if case["bias"]:
        u = u + s["bias"].float()
    y = _act(u, case["act"])[0]
    if case["residual"]:
        y = y + s["residual"].float()
    out = {"y": y.to(torch.bfloat16)}
    if not case["train"]:
        return out
    # the backward pass starts from what the forward pass kept
    out["u"] = u.to(torch.bfloat16)
    du = s["dy"].float() * _act(out["u"].float(), case["act"])[1]
    out["dx"] = (du @ W.t().contiguous()).to(torch.bfloat16)
    out["dW"] = (x.t().contiguous() @ du).to(torch.bfloat16)
    if case["bias"]:
        out["dbias"] = du.sum(dim=0).to(torch.bfloat16)
    return out


_M32 = 0xFFFFFFFF


def _mix(x):
    """int64 values of 32 bits, mixed by multiplications and shifts."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & _M32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & _M32
    return x ^ (x >> 16)


def _random16(n, tensor, t, dev):
    key = _mix((SEED + _mix((t.long() * 0x9E3779B9 + tensor) & _M32)) & _M32)
    i = torch.arange(n, device=dev)
    r = _mix((((i & _M32) + key) & _M32) ^ (((i >> 32) * 0x9E3779B9) & _M32))
    return r & 0xFFFF, r >> 16


def _decode(codes, scale, n):
    x = torch.nn.functional.pad(codes.float(), (0, _up(n, 128) - n)).view(-1, 128)
    return (x.double() * _pow2(scale.to(torch.int32) - 127)[:, None]).reshape(-1)[:n]


def _encode(x, rand, top, mantissa, lowest, keep):
    """Codes' values over their scale and the scale bytes of float64 x; `lowest` the exponent of the smallest normal."""
    n = x.numel()
    pad = _up(n, 128) - n
    b, rand = (torch.nn.functional.pad(t, (0, pad)).view(-1, 128) for t in (x, rand))
    big, e = torch.frexp(b.abs().amax(dim=1))  # big 2^e, big in [0.5, 1); top = 0.875 2^te
    e = e - int(math.frexp(top)[1]) + (big > math.frexp(top)[0]).to(torch.int32)
    e = torch.where(big == 0, torch.full_like(e, -120), e.clamp(-120, 120))
    b = b * _pow2(-e)[:, None]
    s = _pow2((torch.frexp(b.abs())[1] - 1).clamp(min=lowest) - mantissa)
    q = torch.floor((torch.floor(b.abs() / s * 65536.0) + rand) / 65536.0) * s  # by whole numbers: b / s + r / 65536 would round
    if keep:
        q = torch.where((q == 0) & (b != 0), s, q)
    return torch.copysign(q, b).reshape(-1)[:n], (e + 127).to(torch.uint8)


def _plain_adamw(s):
    dev = s["counter"].device
    out = {}
    scale = None
    if s["max_norm"] is not None:
        norm = torch.sqrt(sum(t.double().square().sum() for t in s["grad"]))
        out["norm"] = norm.float().reshape(1)
        # rounded like the norm itself: the step reads it in 32 bits
        scale = (s["max_norm"] / torch.clamp(norm, min=s["max_norm"])).float()
    t = s["counter"][0] + 1
    c1, c2 = 1.0 - BETA1 ** t.double(), 1.0 - BETA2 ** t.double()
    for j in range(len(s["param"])):
        n, eight = s["param"][j].numel(), s["m_scale"][j] is not None
        p = s["param"][j] if s["master"][j] is None else s["master"][j]
        g = s["grad"][j].double()
        g = g if scale is None else g * scale.double()
        m = _decode(s["m"][j], s["m_scale"][j], n) if eight else s["m"][j].double()
        v = _decode(s["v"][j], s["v_scale"][j], n) if eight else s["v"][j].double()
        m = BETA1 * m + (1.0 - BETA1) * g
        v = BETA2 * v + (1.0 - BETA2) * g * g
        step = (m.float() / c1.float()) / (torch.sqrt(v.float() / c2.float()) + ADAM_EPS)
        p.copy_(p - LR * (step + DECAY * p))
        if s["master"][j] is not None:
            s["param"][j].copy_(p)
        if eight:
            rm, rv = _random16(n, j, t, dev)
            q, e = _encode(m, rm, 448.0, 3, -6, False)
            s["m"][j].copy_(q)
            s["m_scale"][j].copy_(e)
            q, e = _encode(v, rv, 57344.0, 2, -14, True)
            s["v"][j].copy_(q)
            s["v_scale"][j].copy_(e)
        else:
            s["m"][j].copy_(m)
            s["v"][j].copy_(v)
    s["counter"][0] += 1
    return _adamw_out(s, out)


def _adamw_out(s, out):
    f = s["flat"]
    out.update(steps=s["counter"], bf16=f["bf16"], f32=f["f32"], master=f["master"], m32=f["m32"], v32=f["v32"], m8=f["m8"],
               v8=f["v8"], m_scale=f["ms"].view(torch.float8_e8m0fnu), v_scale=f["vs"].view(torch.float8_e8m0fnu))
    return out


# ---------------------------------------------------------------- the library's calls

def _plan(s):
    """What a program makes once per shape: the problem, the outputs and the workspaces, or the optimizer."""
    import sparse_mixture_experts_route_amd as moe
    case = s["case"]

    def new(shape, dtype):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    if case["op"] == "adamw":
        opt = moe.AdamW(s["param"], lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=DECAY, max_norm=s["max_norm"],
                        seed=SEED, state={k: s[k] for k in ("master", "m", "m_scale", "v", "v_scale", "counter")})
        s["plan"] = opt
        return opt
    T = case["T"]
    if case["op"] == "linear":
        K, N, train = case["K"], case["N"], case["train"]
        p = moe.make_problem(T, K, 1, 1, N, torch.bfloat16)
        act = {"none": moe.MOET_ACT_NONE, "gelu": moe.MOET_ACT_GELU, "silu": moe.MOET_ACT_SILU,
               "relu": moe.MOET_ACT_RELU}[case["act"]]
        o = {"y": new((T, N), torch.bfloat16)}
        ws = new((moe.moet_workspace_size(p, moe.MOET_STAGE_LINEAR),), torch.uint8)
        if train:
            o.update(u=new((T, N), torch.bfloat16), dx=new((T, K), torch.bfloat16), dW=new((K, N), torch.bfloat16))
            if case["bias"]:
                o["dbias"] = new((N,), torch.bfloat16)
            ws = (ws, new((moe.moet_workspace_size(p, moe.MOET_STAGE_LINEAR_BACKWARD),), torch.uint8))
        s["plan"] = (moe, p, act, o, ws)
        return s["plan"]
    d, E, k, dt = case["d"], case["E"], case["k"], s["x"].dtype
    p = moe.make_problem(T, d, E, k, 64, dt)
    o = {"counts": new((E,), torch.int32), "offsets": new((E + 1,), torch.int32), "perm": new((T * k,), torch.int32),
         "inv": new((T * k,), torch.int32), "x_perm": new((T * k, d), dt), "y": new((T, d), dt)}
    if case["train"]:
        o.update(dy_perm=new((T * k, d), dt), dx=new((T, d), dt), dgate=new((T, k), torch.float32),
                 dlogits=new((T, E), torch.float32))
    ws = new((moe.moet_workspace_size(p, moe.MOET_STAGE_DISPATCH),), torch.uint8)
    s["plan"] = (moe, p, o, ws)
    return s["plan"]


def _own(s):
    plan, case = s.get("plan") or _plan(s), s["case"]
    if case["op"] == "adamw":
        out = {}
        norm = plan.step(s["grad"])
        if norm is not None:
            out["norm"] = norm
        return _adamw_out(s, out)
    if case["op"] == "linear":
        moe, p, act, o, ws = plan
        if not case["train"]:
            moe.moet_linear(p, s["x"], s["W"], s["bias"], act, s["residual"], None, o["y"], ws)
        else:
            moe.moet_linear(p, s["x"], s["W"], s["bias"], act, s["residual"], o["u"], o["y"], ws[0])
            moe.moet_linear_backward(p, s["x"], s["W"], o["u"], act, s["dy"], o["dx"], o["dW"], o.get("dbias"), ws[1])
        return dict(o)
    moe, p, o, ws = plan
    w_in, w_out = (s["gate"], None) if case["early"] else (None, s["gate"])
    moe.moet_dispatch(p, s["idx"], w_in, s["x"], o["counts"], o["offsets"], o["perm"], o["inv"], o["x_perm"], ws)
    moe.moet_combine(p, s["y_perm"], o["inv"], w_out, s["residual"], o["y"])
    if case["train"]:
        early = case["early"]
        moe.moet_combine_backward(p, s["dy"], o["inv"], None if early else s["y_perm"], w_out, o["dy_perm"],
                                  None if early else o["dgate"])
        moe.moet_dispatch_backward(p, s["dx_perm"], o["inv"], s["x"] if early else None, w_in, s["dh"], o["dx"],
                                   o["dgate"] if early else None)
        moe.moet_gate_backward(p, s["logits"], s["idx"], o["dgate"], None, o["dlogits"])
    return dict(o)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_tokens(state) if op == "tokens" else _plain_linear(state) if op == "linear" else _plain_adamw(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_tokens(s):
    case, D = s["case"], torch.float64
    T, d, E, k, dev = case["T"], case["d"], case["E"], case["k"], s["x"].device
    idx = s["idx"].reshape(-1)
    groups = [torch.nonzero(idx == e).reshape(-1) for e in range(E)]
    sel = torch.cat(groups)  # the selection of each row
    counts = torch.tensor([g.numel() for g in groups])
    offsets = torch.tensor([sum(counts[:e].tolist()) for e in range(E + 1)])
    n, R = sel.numel(), T * k
    perm, inv = torch.zeros(R, dtype=torch.int64, device=dev), torch.full((R,), -1, dtype=torch.int64, device=dev)
    perm[:n] = torch.div(sel, k, rounding_mode="floor")
    inv[sel] = torch.arange(n, device=dev)
    gate = s["gate"].reshape(-1).to(D)

    def rows(t, weighted):
        o = torch.zeros((R, d), dtype=D, device=dev)
        o[:n] = t.to(D)[perm[:n]]
        if weighted:
            o[:n] *= gate[sel][:, None]
        return o

    def back(r, weighted, add):
        o = add.to(D).clone()
        src = r[:n].to(D)
        return o.index_add_(0, perm[:n], src * gate[sel][:, None] if weighted else src)

    def dots(r, t):
        o = torch.zeros(R, dtype=D, device=dev)
        o[sel] = (r[:n].to(D) * t.to(D)[perm[:n]]).sum(dim=1)
        return o.view(T, k)

    early = case["early"]
    out = {"counts": counts, "offsets": offsets, "inv": inv, "perm": perm, "x_perm": rows(s["x"], early),
           "y": back(s["y_perm"], not early, s["residual"])}
    if case["train"]:
        out["dy_perm"] = rows(s["dy"], not early)
        out["dx"] = back(s["dx_perm"], early, s["dh"])
        out["dgate"] = dots(s["dx_perm"], s["x"]) if early else dots(s["y_perm"], s["dy"])
        p = torch.softmax(s["logits"].to(D), dim=1)
        dp = torch.zeros((T, E), dtype=D, device=dev)
        dp.view(-1).index_add_(0, perm[:n] * E + idx[sel].long(), out["dgate"].reshape(-1)[sel])
        out["dlogits"] = p * dp - p * (p * dp).sum(dim=1, keepdim=True)
    return out


def _exact_linear(s):
    case, D = s["case"], torch.float64
    W, x = s["W"].to(D), s["x"].to(D)
    u = torch.matmul(x, W)
    if case["bias"]:
        u += s["bias"].to(D)[None, :]

    def value(z):
        if case["act"] == "gelu":
            return z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
        return {"none": lambda: z, "relu": lambda: z.clamp(min=0.0), "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()

    out = {"y": value(u) + s["residual"].to(D) if case["residual"] else value(u)}
    if not case["train"]:
        return out
    out["u"] = u
    z = u.to(torch.bfloat16).to(D)
    if case["act"] == "gelu":
        a = math.sqrt(8.0 / math.pi)
        h = torch.sigmoid(a * (z + 0.044715 * z ** 3))
        slope = h + z * h * (1.0 - h) * a * (1.0 + 3 * 0.044715 * z ** 2)
    elif case["act"] == "silu":
        h = torch.sigmoid(z)
        slope = h + z * h * (1.0 - h)
    else:
        slope = torch.ones_like(z) if case["act"] == "none" else torch.heaviside(z, torch.zeros((), dtype=D, device=z.device))
    du = slope * s["dy"].to(D)
    out["dx"] = torch.matmul(du, W.t().contiguous())
    out["dW"] = torch.matmul(x.t().contiguous(), du)
    if case["bias"]:
        out["dbias"] = du.sum(dim=0)
    return out


def _exact_codes(x, rand, top, mantissa, lowest, keep):
    """Values over the scale, and scales, of rows of 128 float64 values; spacings from the bits of the number."""
    b, scale = torch.zeros((_up(x.numel(), 128),), dtype=torch.float64, device=x.device), None
    b[:x.numel()] = x
    rnd = torch.zeros(b.shape, dtype=torch.int64, device=x.device)
    rnd[:x.numel()] = rand
    b, rnd = b.view(-1, 128), rnd.view(-1, 128)
    e = torch.full((b.shape[0],), -120.0, dtype=torch.float64, device=x.device)
    for trial in range(119, -121, -1):  # the smallest that holds the row
        e = torch.where((b.abs().amax(dim=1) > top * 2.0 ** trial) & (e < trial + 1), torch.full_like(e, trial + 1), e)
    scale = torch.exp2(e)
    b = b / scale[:, None]
    exponent = (b.abs().view(torch.int64) >> 52) - 1023
    s = torch.exp2((exponent.clamp(min=lowest) - mantissa).to(torch.float64))
    units = (b.abs() / s * 65536.0).floor().to(torch.int64) + rnd  # r / 65536 is whole in these units
    q = (units >> 16).to(torch.float64)
    if keep:
        q[(q == 0) & (b > 0)] = 1.0
    return (torch.sign(b) * q * s).reshape(-1)[:x.numel()], scale


def _exact_adamw(s):
    D = torch.float64
    flat = {k: (t.to(D) if t.dtype != torch.uint8 else torch.exp2(t.to(D) - 127.0)) for k, t in s["flat"].items()}
    out = {}
    scale = 1.0
    if s["max_norm"] is not None:
        norm = math.sqrt(math.fsum(float(t.to(D).pow(2).sum()) for t in s["grad"]))
        out["norm"] = torch.tensor([norm], dtype=D)
        scale = float(torch.tensor(min(1.0, s["max_norm"] / norm), dtype=torch.float32)) if norm else 1.0
    t = STEPS + 1
    k1, k2 = -math.expm1(t * math.log(BETA1)), -math.expm1(t * math.log(BETA2))
    at = {"bf16": 0, "f32": 0, 32: 0, 8: 0, "s": 0}
    for j, (n, dt, bits) in enumerate(_sizes(s["case"])):
        a, b, c, nb = at[dt], at[bits], at["s"], (n + 127) // 128
        at[dt] += nb * 128
        at[bits] += nb * 128
        p = flat["master" if dt == "bf16" else "f32"][a:a + n]
        g = s["grad"][j].to(D) * scale
        m, v = flat["m%d" % bits][b:b + n], flat["v%d" % bits][b:b + n]
        if bits == 8:
            at["s"] += (nb + 255) // 256 * 256
            m = m * flat["ms"][c:c + nb].repeat_interleave(128)[:n]
            v = v * flat["vs"][c:c + nb].repeat_interleave(128)[:n]
        m = m * BETA1 + g * (1.0 - BETA1)
        v = v * BETA2 + g * g * (1.0 - BETA2)
        p -= LR * (m / k1 / ((v / k2).sqrt() + ADAM_EPS) + DECAY * p)
        if dt == "bf16":
            flat["bf16"][a:a + n] = p
        if bits == 32:
            flat["m32"][b:b + n], flat["v32"][b:b + n] = m, v
            continue
        key = _exact_mix(SEED + _exact_mix(t * 0x9E3779B9 + j))
        lanes = torch.arange(n, device=m.device)  # fewer than 2^32: no high half
        r = _exact_mix(lanes + key)
        flat["m8"][b:b + n], flat["ms"][c:c + nb] = _exact_codes(m, r % 65536, 448.0, 3, -6, False)
        flat["v8"][b:b + n], flat["vs"][c:c + nb] = _exact_codes(v, r // 65536, 57344.0, 2, -14, True)
    out.update(steps=torch.tensor([t, 0]), bf16=flat["bf16"], f32=flat["f32"], master=flat["master"], m32=flat["m32"],
               v32=flat["v32"], m8=flat["m8"], v8=flat["v8"], m_scale=flat["ms"], v_scale=flat["vs"])
    return out


def _exact_mix(x):
    """The generator's mixing of the low 32 bits of a whole number or of an int64 tensor of them."""
    x = x % (1 << 32)
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        x = x ^ (x // (1 << shift))
        # by halves, so that products stay inside 63 bits
        x = (x * (factor % 65536) + (x * (factor // 65536) % 65536) * 65536) % (1 << 32)
    return x ^ (x // (1 << 16))


def exact(case, seed):
    s = prepare(case, seed)
    return {"tokens": _exact_tokens, "linear": _exact_linear, "adamw": _exact_adamw}[case["op"]](s)
