"""Measured cases of the block operators around the sparse mixture-of-experts layer.

Three operators, each with a plain form (elementary torch operations in
float32) and the library's own calls:

  norm      h = x + residual, y = h * rsqrt(mean(h^2) + eps) * gain, and y in
            8 bits; in training also the backward pass
  balance   the router's load-balancing loss, the per-expert counts and the
            gradient of the logits
  experts   the expert FFNs over ragged row groups with rows, hidden
            activations and weights in 8 bits

The 8-bit format: 128 values along the contraction share a scale 2^e, e the
smallest integer with max|v| <= 448 * 2^e (kept in [-120, 120]) and held as the
byte e + 127; a value is its e4m3 code times the scale. Rows are padded with
zero codes to a multiple of 128 and their scales to a multiple of 16 bytes.
Expert weights are laid out once for the matrix cores, as
[expert][column / 32][k / 128][16-byte piece pair 4][2][column % 32][16], with
scales [expert][column / 32][k / 128][column % 32].
"""

import math

import torch

own = False

EPS = 1e-6
COEF = 0.01


# ---------------------------------------------------------------- the cases

def _norm(name, T, d, dtype, residual, train):
    return {"name": name, "op": "norm", "T": T, "d": d, "dtype": dtype, "residual": residual, "train": train}


def _balance(name, T, E, k, skew, masked):
    return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "skew": skew, "masked": masked}


def _experts(name, T, d, E, k, de, skew):
    return {"name": name, "op": "experts", "T": T, "d": d, "E": E, "k": k, "de": de, "skew": skew}


def listed():
    return [
        # one decode step of eight sequences in front of a 7168-wide layer: latency counts
        _norm("norm_decode_8x7168", 8, 7168, "bf16", True, False),
        # a prefill in front of the large sparse layer: the copy rate counts
        _norm("norm_16384x7168", 16384, 7168, "bf16", True, False),
        # a training step in front of the fine-grained layer, both directions
        _norm("norm_train_8192x2048", 8192, 2048, "bf16", True, True),
        # an odd number of rows of an odd multiple of 64 in float32, both directions
        _norm("norm_train_777x320_f32", 777, 320, "f32", True, True),
        # the router of the tiny layer: launch latency
        _balance("balance_64x8", 64, 8, 2, 0.0, False),
        # the router of the fine-grained layer
        _balance("balance_8192x64", 8192, 64, 8, 0.0, False),
        # the router of the large sparse layer over a padded batch with favoured experts
        _balance("balance_16384x256_masked", 16384, 256, 8, 1.0, True),
        # one token through a fine-grained layer: eight experts' weights are streamed
        _experts("experts_decode_1x2048", 1, 2048, 64, 8, 1024, 0.0),
        # a decode batch of 32 through coarse experts
        _experts("experts_decode_32x2048", 32, 2048, 8, 2, 8192, 0.0),
        # ragged groups at odd widths, some of them empty
        _experts("experts_ragged_777x320", 777, 320, 12, 3, 448, 3.0),
        # the fine-grained layer at its full batch
        _experts("experts_8192x2048", 8192, 2048, 64, 8, 1024, 0.0),
        # the coarse layer at its full batch
        _experts("experts_4096x2048_coarse", 4096, 2048, 8, 2, 8192, 0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("norm", "balance", "experts"))
    if op == "norm":
        train = rng.random() < 0.5
        d = 64 * _log_int(rng, 1, 112)
        T = min(_log_int(rng, 1, 16384), (1 << 25) // d if train else 16384)
        return {"op": op, "T": T, "d": d, "dtype": rng.choice(("bf16", "bf16", "f32")), "residual": rng.random() < 0.7,
                "train": train}
    if op == "balance":
        E = _log_int(rng, 2, 256)
        return {"op": op, "T": _log_int(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 8)),
                "skew": rng.choice((0.0, 1.0, 3.0)), "masked": rng.random() < 0.5}
    E = _log_int(rng, 1, 64)
    k = rng.randint(1, min(E, 8))
    return {"op": op, "T": _log_int(rng, 1, 4096), "d": 64 * _log_int(rng, 1, 32), "E": E, "k": k,
            "de": 64 * _log_int(rng, 1, 32), "skew": rng.choice((0.0, 1.0, 3.0))}


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        d, es = case["d"], 2 if case["dtype"] == "bf16" else 4
        adds = 1 if case["residual"] else 0
        if case["train"]:
            # forward: x, residual in; h (when added), y out. backward: h, dy, dh in; dx out
            return {"bytes": T * d * es * (6 + 2 * adds) + 2 * d * es + d * 4, "flops": 20 * T * d}
        return {"bytes": T * d * (es * (2 + 2 * adds) + 1) + d * es + T * d // 128, "flops": 8 * T * d}
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        return {"bytes": 8 * T * E + 4 * T * k + 8 * E, "flops": 12 * T * E}
    d, E, k, de = case["d"], case["E"], case["k"], case["de"]
    busy = min(E, T * k)
    return {"bytes": T * d + 4 * T * k + 2 * busy * d * de + 2 * T * k * d, "flops": 4 * T * k * d * de}


# ---------------------------------------------------------------- inputs

def _up(n, m):
    return (n + m - 1) // m * m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _router_logits(g, T, E, skew):
    logits = torch.randn((T, E), generator=g, device="cuda")
    return (logits + skew * torch.randn((E,), generator=g, device="cuda")).contiguous()


def _topk(logits, k):
    """Descending logits, ties to the lower index."""
    return torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()


def _encode(v):
    """float32 rows [..., K] (K a multiple of 128) to (codes [..., K] e4m3, scale bytes [..., K / 128] uint8)."""
    b = v.reshape(*v.shape[:-1], -1, 128)
    m, e = torch.frexp(b.abs().amax(dim=-1))  # max = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875).to(torch.int32)).clamp(-120, 120)
    e = torch.where(m == 0, torch.full_like(e, -120), e)
    codes = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes.reshape(v.shape), (e + 127).to(torch.uint8)


def _pad(v, n):
    """Zeros behind the last axis, up to n."""
    return v if v.shape[-1] == n else torch.nn.functional.pad(v, (0, n - v.shape[-1]))


def _weights(g, E, K, N, std):
    """Quantised expert weights [E, K, N] in the matrix-core layout."""
    Kp = _up(K, 128)
    w = _pad(_normal(g, (E, N, K), std, torch.bfloat16).float(), Kp)
    codes, scale = _encode(w)
    codes = codes.view(torch.uint8).view(E, N // 32, 32, Kp // 128, 4, 2, 16).permute(0, 1, 3, 4, 5, 2, 6).contiguous()
    return codes, scale.view(E, N // 32, 32, Kp // 128).permute(0, 1, 3, 2).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    T = case["T"]
    s = {"case": case}
    if case["op"] == "norm":
        d, dt = case["d"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"] = _normal(g, (T, d), 1.0, dt)
        s["residual"] = _normal(g, (T, d), 2.0, dt) if case["residual"] else None
        s["gain"] = (1.0 + 0.1 * torch.randn((d,), generator=g, device="cuda")).to(dt)
        if case["train"]:
            s["dy"] = _normal(g, (T, d), 1.0, dt)
            s["dh"] = _normal(g, (T, d), 1.0, dt)
        return s
    E, k = case["E"], case["k"]
    logits = _router_logits(g, T, E, case["skew"])
    idx = _topk(logits, k)
    if case["op"] == "balance":
        s["logits"], s["idx"] = logits, idx
        # a padded batch: about an eighth of the tokens are padding
        s["mask"] = (torch.rand((T,), generator=g, device="cuda") < 0.875).to(torch.uint8) if case["masked"] else None
        return s
    d, de = case["d"], case["de"]
    flat = idx.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    s["perm"] = (order // k).to(torch.int32)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["cap"] = int(counts.max())
    x = _pad(_normal(g, (T, d), 1.0, torch.bfloat16).float(), _up(d, 128))
    codes, scale = _encode(x)
    s["x8"], s["x_scale"] = codes, _pad(scale, _up(scale.shape[1], 16)).contiguous()
    s["W1q"], s["W1s"] = _weights(g, E, d, de, d ** -0.5)
    s["W2q"], s["W2s"] = _weights(g, E, de, d, de ** -0.5)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_norm(s):
    case, x = s["case"], s["x"]
    dt, d = x.dtype, case["d"]
    h = (x.float() + s["residual"].float()).to(dt) if case["residual"] else x
    hf, gain = h.float(), s["gain"].float()
    rstd = 1.0 / torch.sqrt(hf.square().mean(dim=1) + EPS)
    z = hf * rstd[:, None]
    y = z * gain
    out = {"y": y.to(dt), "rstd": rstd}
    if case["residual"]:
        out["h"] = h
    if not case["train"]:
        codes, scale = _encode(_pad(y, _up(d, 128)))
        out["y8"], out["scale"] = codes, _pad(scale, _up(scale.shape[1], 16)).contiguous().view(torch.float8_e8m0fnu)
        return out
    a = s["dy"].float() * gain
    out["dx"] = (rstd[:, None] * (a - z * (a * z).mean(dim=1, keepdim=True)) + s["dh"].float()).to(dt)
    out["dgain"] = (s["dy"].float() * z).sum(dim=0)
    return out


def _plain_balance(s):
    case, logits, idx = s["case"], s["logits"], s["idx"].long()
    T, E, k = case["T"], case["E"], case["k"]
    valid = s["mask"] != 0 if s["mask"] is not None else torch.ones((T,), dtype=torch.bool, device=logits.device)
    n = valid.sum()
    hits = (idx[:, :, None] == torch.arange(E, device=logits.device)).sum(dim=1)
    counts = (hits * valid[:, None]).sum(dim=0)
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    p = e / e.sum(dim=1, keepdim=True) * valid[:, None]
    some = n.clamp(min=1).double()
    f = counts.double() / (some * k)
    mean_prob = (p.sum(dim=0, dtype=torch.float64) / some).float()
    loss = (COEF * E * (f * mean_prob.double()).sum()).float()
    # f_e - sum f p does not change when all f move by the same amount: taken from the row's most
    # probable expert, whose own term then has no large parts that cancel
    c = ((counts - counts[logits.argmax(dim=1)][:, None]).double() / (some * k)).float()
    dlogits = (COEF * E / some).float() * p * (c - (p * c).sum(dim=1, keepdim=True))
    return {"loss": loss.reshape(1), "counts": counts.to(torch.int32), "mean_prob": mean_prob, "dlogits": dlogits}


def _decode(codes, scale):
    """codes [..., K] e4m3, scale bytes [..., K / 128]: float32 values."""
    b = codes.float().reshape(*codes.shape[:-1], -1, 128)
    return torch.ldexp(b, scale.to(torch.int32).unsqueeze(-1) - 127).reshape(codes.shape)


def _decode_weights(q, ws):
    """Float32 [E, Kp, N] from the matrix-core layout."""
    E, NG, KB = q.shape[0], q.shape[1], q.shape[2]
    codes = q.permute(0, 1, 5, 2, 3, 4, 6).reshape(E, NG * 32, KB * 128).view(torch.float8_e4m3fn)
    scale = ws.permute(0, 1, 3, 2).reshape(E, NG * 32, KB)
    return _decode(codes, scale).transpose(1, 2).contiguous()


def _plain_experts(s):
    case = s["case"]
    E, k, cap, d = case["E"], case["k"], s["cap"], case["d"]
    offsets, perm = s["offsets"].long(), s["perm"].long()
    R = case["T"] * k
    r = torch.arange(R, device=perm.device)
    e = torch.searchsorted(offsets[1:], r, right=True)
    slot = e * cap + r - offsets[e]
    dp = s["x8"].shape[1]
    x = _decode(s["x8"], s["x_scale"][:, :dp // 128])
    xe = torch.zeros((E * cap, dp), device=x.device)
    xe[slot] = x[perm]
    u = torch.bmm(xe.view(E, cap, dp), _decode_weights(s["W1q"], s["W1s"]))
    u = 0.5 * u * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (u + 0.044715 * u * u * u)))
    codes, scale = _encode(_pad(u, _up(case["de"], 128)))
    y = torch.bmm(_decode(codes, scale), _decode_weights(s["W2q"], s["W2s"]))
    return {"y_perm": y.view(E * cap, d)[slot].to(torch.bfloat16)}


# ---------------------------------------------------------------- the library's calls

def _plan(s):
    """What a program allocates once per shape: the problem, the outputs, the workspace."""
    import sparse_mixture_experts_route_amd as moe
    case = s["case"]
    T = case["T"]

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if case["op"] == "norm":
        d, dt = case["d"], s["x"].dtype
        p = moe.make_problem(T, d, 1, 1, 64, dt)
        o = {"h": new((T, d), dt) if case["residual"] else None, "y": new((T, d), dt), "rstd": new((T,), torch.float32)}
        if case["train"]:
            o["dx"], o["dgain"] = new((T, d), dt), new((d,), torch.float32)
            ws = new((moe.moex_workspace_size(p, moe.MOEX_STAGE_NORM_BACKWARD),), torch.uint8)
        else:
            kb = _up(d, 128) // 128
            o["y8"], o["scale"] = new((T, kb * 128), torch.float8_e4m3fn), new((T, _up(kb, 16)), torch.uint8)
            ws = None
    elif case["op"] == "balance":
        E = case["E"]
        p = moe.make_problem(T, 64, E, case["k"], 64, torch.float32)
        o = {"loss": new((1,), torch.float32), "counts": new((E,), torch.int32), "mean_prob": new((E,), torch.float32),
             "dlogits": new((T, E), torch.float32)}
        ws = new((moe.moex_workspace_size(p, moe.MOEX_STAGE_BALANCE),), torch.uint8)
    else:
        p = moe.make_problem(T, case["d"], case["E"], case["k"], case["de"], torch.bfloat16)
        o = {"y_perm": new((T * case["k"], case["d"]), torch.bfloat16)}
        ws = new((moe.moex_workspace_size(p, moe.MOEX_STAGE_FFN_FP8),), torch.uint8)
    s["plan"] = (moe, p, o, ws)
    return s["plan"]


def _own(s):
    moe, p, o, ws = s.get("plan") or _plan(s)
    case = s["case"]
    if case["op"] == "norm":
        h = o["h"] if case["residual"] else s["x"]
        if case["train"]:
            moe.moex_add_rmsnorm(p, s["x"], s["residual"], s["gain"], EPS, o["h"], o["y"], None, None, o["rstd"])
            moe.moex_add_rmsnorm_backward(p, h, s["gain"], o["rstd"], s["dy"], s["dh"], o["dx"], o["dgain"], ws)
            out = {"y": o["y"], "rstd": o["rstd"], "dx": o["dx"], "dgain": o["dgain"]}
        else:
            moe.moex_add_rmsnorm(p, s["x"], s["residual"], s["gain"], EPS, o["h"], o["y"], o["y8"], o["scale"],
                                 o["rstd"])
            out = {"y": o["y"], "rstd": o["rstd"], "y8": o["y8"], "scale": o["scale"].view(torch.float8_e8m0fnu)}
        if case["residual"]:
            out["h"] = o["h"]
        return out
    if case["op"] == "balance":
        moe.moex_balance_loss(p, s["logits"], s["idx"], s["mask"], COEF, o["loss"], o["counts"], o["mean_prob"],
                              o["dlogits"], ws)
        return dict(o)
    moe.moex_grouped_ffn_fp8(p, s["x8"], s["x_scale"], s["perm"], s["offsets"], s["W1q"], s["W1s"], s["W2q"], s["W2s"],
                             o["y_perm"], ws)
    return dict(o)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_norm(state) if op == "norm" else _plain_balance(state) if op == "balance" else _plain_experts(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3_64(v):
    """Nearest e4m3 value, ties to even, of float64 values of at most 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _blocks_64(v):
    """(codes, scales) of float64 rows whose width is a multiple of 128."""
    b = v.reshape(*v.shape[:-1], -1, 128)
    top = b.abs().amax(dim=-1)
    e = torch.ceil(torch.log2(top / 448.0).clamp(min=-120.0))
    e = torch.where(torch.exp2(e - 1) * 448.0 >= top, e - 1, e)  # should the logarithm have rounded up
    e = torch.where(torch.exp2(e) * 448.0 < top, e + 1, e).clamp(-120.0, 120.0)
    scale = torch.exp2(e)
    return _e4m3_64(b / scale[..., None]).reshape(v.shape), scale


def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    if case["op"] == "norm":
        x, g = s["x"].to(D), s["gain"].to(D)
        h = (x + s["residual"].to(D)).to(s["x"].dtype).to(D) if case["residual"] else x
        rstd = (h.pow(2).sum(dim=1) / case["d"] + EPS).rsqrt()
        z = h * rstd[:, None]
        out = {"y": z * g, "rstd": rstd}
        if case["residual"]:
            out["h"] = h
        if not case["train"]:
            codes, scale = _blocks_64(_pad(out["y"], _up(case["d"], 128)))
            out["y8"] = codes
            out["scale"] = torch.nn.functional.pad(scale, (0, _up(scale.shape[1], 16) - scale.shape[1]),
                                                   value=2.0 ** -127)
            return out
        dy = s["dy"].to(D)
        a = dy * g
        out["dx"] = rstd[:, None] * (a - z * ((a * z).sum(dim=1, keepdim=True) / case["d"])) + s["dh"].to(D)
        out["dgain"] = (dy * z).sum(dim=0)
        return out
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        rows = torch.nonzero(s["mask"]).reshape(-1) if s["mask"] is not None else torch.arange(case["T"], device="cuda")
        n = rows.numel()
        counts = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=E)
        dlogits = torch.zeros((case["T"], E), dtype=D, device="cuda")
        if n == 0:
            return {"loss": torch.zeros(1, dtype=D), "counts": counts, "mean_prob": torch.zeros(E, dtype=D),
                    "dlogits": dlogits}
        p = torch.softmax(s["logits"][rows].to(D), dim=1)
        f = counts.to(D) / (n * k)
        shift = (counts * E - n * k).to(D) / (float(n) * k * E)  # f less an even share: the same gradient
        dlogits[rows] = COEF * E / n * p * (shift[None, :] - (p @ shift)[:, None])
        P = p.mean(dim=0)
        return {"loss": (COEF * E * torch.dot(f, P)).reshape(1), "counts": counts, "mean_prob": P, "dlogits": dlogits}
    d, de, E = case["d"], case["de"], case["E"]

    def rows64(codes, scale):
        return codes.to(D) * torch.exp2(scale[:, :codes.shape[1] // 128].to(D) - 127).repeat_interleave(128, dim=1)

    def weights64(q, ws, e):
        c = q[e].permute(0, 4, 1, 2, 3, 5).reshape(-1, q.shape[2] * 128).view(torch.float8_e4m3fn)
        return rows64(c, ws[e].permute(0, 2, 1).reshape(c.shape[0], -1)).t().contiguous()

    x = rows64(s["x8"], s["x_scale"])
    y = torch.zeros((case["T"] * case["k"], d), dtype=D, device="cuda")
    lim = s["offsets"].tolist()
    for e in range(E):
        if lim[e] == lim[e + 1]:
            continue
        u = x[s["perm"][lim[e]:lim[e + 1]].long()] @ weights64(s["W1q"], s["W1s"], e)
        h = u * torch.sigmoid(math.sqrt(8.0 / math.pi) * (u + 0.044715 * u ** 3))
        codes, scale = _blocks_64(_pad(h, _up(de, 128)))
        h = codes * scale.repeat_interleave(128, dim=1)
        y[lim[e]:lim[e + 1]] = h @ weights64(s["W2q"], s["W2s"], e)
    return {"y_perm": y}
