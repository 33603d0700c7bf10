"""The router's balance loss, counts and gradient against float64, alone and inside the layer's backward pass."""

import numpy as np
import pytest
import torch

import oracle
from ext_helpers import HALF, assert_within, f64, gen
from gpu_helpers import U32, announce, i64, needs_gpu
from harness import host_array, make_dense, make_inputs, scaled_config
from oracle import block_ops as ob

pytestmark = [pytest.mark.gpu, needs_gpu]


def make(T, E, k, skew, masked, seed):
    g = gen(seed)
    logits = torch.randn((T, E), generator=g, device="cuda") + skew * torch.randn((E,), generator=g, device="cuda")
    idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
    mask = (torch.rand((T,), generator=g, device="cuda") < 0.7).to(torch.uint8) if masked else None
    return logits, idx, mask


def call(moe, logits, idx, mask, coef, dlogits=True, stream=None):
    T, E = logits.shape
    p = moe.make_problem(T, 64, E, idx.shape[1], 64, torch.float32)
    o = {"loss": torch.full((1,), 7.0, device="cuda"), "counts": torch.full((E,), -7, dtype=torch.int32, device="cuda"),
         "mean_prob": torch.full((E,), 7.0, device="cuda"),
         "dlogits": torch.full((T, E), 7.0, device="cuda") if dlogits else None}
    ws = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_BALANCE), dtype=torch.uint8, device="cuda")
    moe.moex_balance_loss(p, logits, idx, mask, coef, o["loss"], o["counts"], o["mean_prob"], o["dlogits"], ws, stream)
    return o


def check(logits, idx, mask, coef, o):
    l64 = f64(logits)
    T, E = l64.shape
    k = idx.shape[1]
    ref = ob.balance_loss(l64, i64(idx), None if mask is None else mask.cpu().numpy(), float(np.float32(coef)))
    assert np.array_equal(ref["counts"], i64(o["counts"]))
    valid = np.ones(T, bool) if mask is None else mask.cpu().numpy() != 0
    n = max(int(valid.sum()), 1)
    # p: the difference from the row's maximum is off by 2^-24 of itself, the exponential by 2 units,
    # the sum by at most E units, the division and its product by one each
    top = np.where(np.isneginf(l64.max(axis=1, keepdims=True)), 0.0, l64.max(axis=1, keepdims=True))
    far = np.where(np.isneginf(l64), 0.0, np.abs(l64 - top))
    dp = (np.minimum(far, 110.0) + E + 5) * U32 * ref["p"] + 1e-37
    assert_within("mean_prob", f64(o["mean_prob"]), ref["mean_prob"],
                  (dp[valid].sum(axis=0) + (T + 300) * U32 * ref["p"].sum(axis=0)) / n + U32 * ref["mean_prob"])
    f = ref["counts"] / (n * k)
    assert_within("loss", f64(o["loss"])[0:1], np.array([ref["loss"]]),
                  np.array([abs(coef) * E * (f * (dp[valid].sum(axis=0) + (T + 300) * U32 * ref["p"].sum(axis=0))).sum()
                            / n + 4 * U32 * abs(ref["loss"]) + 1e-37]))
    if o["dlogits"] is not None:
        # f from the most probable expert (an exact difference); the bracket's own sum by E + 4 units
        sh = f[None, :] - f[np.argmax(l64, axis=1)][:, None]
        mag = np.abs(sh) + (ref["p"] * np.abs(sh)).sum(axis=1, keepdims=True)
        dsum = (dp * np.abs(sh)).sum(axis=1, keepdims=True)
        w = abs(coef) * E / n
        bound = w * (ref["p"] * ((E + 10) * U32 * mag + dsum) + dp * mag) + 1e-37
        # exact ties for the maximum may be taken from either expert: the same value, other roundings
        bound = bound + w * ref["p"] * (E + 10) * U32 * 2 * f.max()
        assert_within("dlogits", f64(o["dlogits"]), ref["dlogits"], bound)
    return ref


CASES = [  # T, E, k, skew, masked: every lane split, odd E, one expert, k = E, several rounds of workgroups
    (1, 1, 1, 0.0, False), (1, 8, 2, 0.0, True), (64, 8, 2, 0.0, False), (5, 2, 1, 3.0, False), (33, 3, 3, 1.0, True),
    (257, 5, 2, 1.0, False), (100, 17, 4, 0.0, True), (300, 33, 8, 3.0, False), (777, 12, 3, 1.0, True),
    (1000, 64, 8, 0.0, False), (130, 100, 6, 1.0, True), (4099, 160, 8, 1.0, True), (90, 255, 9, 0.0, False),
    (2000, 256, 8, 3.0, True), (20001, 4, 1, 0.0, True), (70000, 16, 2, 1.0, False), (3, 256, 256, 0.0, False),
]


@pytest.mark.parametrize("T,E,k,skew,masked", CASES)
def test_loss_counts_and_gradient(moe, T, E, k, skew, masked):
    announce(f"balance T={T} E={E} k={k} skew={skew} masked={masked}")
    logits, idx, mask = make(T, E, k, skew, masked, 3)
    o = call(moe, logits, idx, mask, 0.01)
    again = call(moe, logits, idx, mask, 0.01)
    only = call(moe, logits, idx, mask, 0.01, dlogits=False)
    torch.cuda.synchronize()
    check(logits, idx, mask, 0.01, o)
    for key in ("loss", "counts", "mean_prob"):
        assert torch.equal(o[key], again[key]) and torch.equal(o[key], only[key])
    assert torch.equal(o["dlogits"], again["dlogits"])


def test_masked_rows_are_not_read(moe):
    """NaN, infinities and wild indices in masked rows change nothing; their gradient is 0."""
    announce("balance masked garbage")
    logits, idx, mask = make(500, 24, 3, 1.0, True, 4)
    clean = call(moe, logits, idx, mask, 0.5)
    dirty_l, dirty_i = logits.clone(), idx.clone()
    rows = (mask == 0).nonzero().reshape(-1)
    dirty_l[rows[0::3]] = float("nan")
    dirty_l[rows[1::3]] = float("inf")
    dirty_l[rows[2::3]] = torch.finfo(torch.float32).min
    dirty_i[rows] = 1 << 30
    dirty = call(moe, dirty_l, dirty_i, mask.bool(), 0.5)
    torch.cuda.synchronize()
    for key in clean:
        assert torch.equal(clean[key], dirty[key]), key
    assert not clean["dlogits"][rows].any()


def test_all_masked(moe):
    announce("balance all masked")
    logits, idx, _ = make(70, 9, 2, 1.0, False, 5)
    o = call(moe, logits, idx, torch.zeros(70, dtype=torch.uint8, device="cuda"), 1.0)
    for key in o:
        assert not o[key].any(), key


def test_infinities_and_foreign_indices(moe):
    announce("balance infinities")
    logits, idx, _ = make(64, 12, 2, 1.0, False, 6)
    logits[:, 5] = float("-inf")          # an expert taken out
    logits[3] = float("-inf")             # a row with no probability at all
    logits[4] = torch.finfo(torch.float32).min  # all at the type's lowest value: even probabilities
    logits[5, 1:] = torch.finfo(torch.float32).min
    idx[7, 0] = -1
    idx[8, 1] = 12
    o = call(moe, logits, idx, None, 0.1)
    torch.cuda.synchronize()
    check(logits, idx, None, 0.1, o)
    out = [t for t in range(64) if t not in (4, 5)]  # rows whose expert 5 is still at -infinity
    assert not o["dlogits"][3].any() and not o["dlogits"][out, 5].any()
    logits[9, 2] = float("nan")  # a NaN of a valid row is seen: in its row, the means and the loss
    logits[10, 3] = float("inf")
    o2 = call(moe, logits, idx, None, 0.1)
    torch.cuda.synchronize()
    assert torch.isnan(o2["dlogits"][9]).all() and torch.isnan(o2["dlogits"][10]).any() and torch.isnan(o2["loss"]).all()
    keep = [t for t in range(64) if t not in (9, 10)]
    assert torch.equal(o2["dlogits"][keep], o["dlogits"][keep])
    assert torch.equal(o2["counts"], o["counts"])


def test_gradient_is_the_difference_quotient(moe):
    """The loss of the same routing at moved logits, taken by the kernel itself in
    float32: a step large enough that the loss's own rounding stays small."""
    announce("balance differences")
    T, E, k, coef, s = 6, 8, 2, 1.0, 2.0 ** -5
    logits, idx, _ = make(T, E, k, 2.0, False, 7)
    o = call(moe, logits, idx, None, coef)
    for t, e in ((0, 0), (1, 5), (5, 7), (3, 2)):
        up, dn = logits.clone(), logits.clone()
        up[t, e] += s
        dn[t, e] -= s
        lu, ld = (float(call(moe, v, idx, None, coef)["loss"]) for v in (up, dn))
        num = (lu - ld) / (2 * s)
        # third derivatives of a softmax term are at most 1 in size: s^2 / 6 of w; the loss rounds at 2^-24
        tol = coef * E / T * s * s / 6 + 4 * U32 * abs(lu) / s
        assert abs(num - float(o["dlogits"][t, e])) <= tol


@pytest.mark.parametrize("T,d,E,k,de,masked", [(300, 256, 16, 4, 320, True), (9, 512, 8, 2, 256, False),
                                               (1024, 256, 64, 8, 128, True)])
def test_backward_balanced(moe, T, d, E, k, de, masked):
    """The layer's backward pass with the loss added: everything that the loss does
    not reach is bit for bit moe_backward's, and the router's gradients are the
    layer's plus the loss's."""
    announce(f"backward balanced T={T} d={d} E={E} k={k} de={de}")
    cfg = scaled_config("skewed", T=T, d_model=d, E=E, k=k, d_expert=de, suffix="balanced")
    inp = make_inputs(cfg, seed=31, device="cuda")
    x, wr, b, W1, W2 = inp["x"], inp["w_router"], inp["router_bias"], inp["W1"], inp["W2"]
    dy = make_dense((T, d), 1.0, seed=31, tag=9, device="cuda")
    mask = (torch.rand((T,), generator=gen(8), device="cuda") < 0.8).to(torch.uint8) if masked else None
    p = moe.make_problem(T, d, E, k, de, x.dtype)
    ws = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_TRAIN_BALANCED), dtype=torch.uint8, device="cuda")
    bf, f32 = torch.bfloat16, torch.float32

    def outs():
        return {"dx": torch.empty((T, d), dtype=bf, device="cuda"), "dwr": torch.empty((d, E), dtype=bf, device="cuda"),
                "db": torch.empty(E, dtype=f32, device="cuda"), "dW1": torch.empty_like(W1), "dW2": torch.empty_like(W2)}

    y = torch.empty_like(x)
    a, c = outs(), outs()
    moe.moe_forward_train(p, x, wr, b, W1, W2, y, ws)
    moe.moe_backward(p, x, wr, W1, W2, dy, a["dx"], a["dwr"], a["db"], a["dW1"], a["dW2"], None, None, ws)
    coef = 20.0  # large enough that the loss's part stands out of the bf16 roundings
    loss, counts, mp = (torch.empty(1, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda"),
                        torch.empty(E, device="cuda"))
    moe.moe_forward_train(p, x, wr, b, W1, W2, y, ws)
    moe.moex_backward_balanced(p, x, wr, W1, W2, dy, mask, coef, c["dx"], c["dwr"], c["db"], c["dW1"], c["dW2"], loss,
                               counts, mp, ws)
    logits, idx, gate = (torch.empty((T, E), device="cuda"), torch.empty((T, k), dtype=torch.int32, device="cuda"),
                         torch.empty((T, k), device="cuda"))
    wsr = torch.empty(moe.moe_workspace_size(p, moe.MOE_STAGE_ROUTE), dtype=torch.uint8, device="cuda")
    moe.moe_route_ws(p, x, wr, b, logits, idx, gate, wsr)
    alone = call(moe, logits, idx, mask, coef)
    torch.cuda.synchronize()
    assert torch.equal(a["dW1"], c["dW1"]) and torch.equal(a["dW2"], c["dW2"])
    assert torch.equal(loss, alone["loss"]) and torch.equal(counts, alone["counts"])
    assert torch.equal(mp, alone["mean_prob"])
    dl = f64(alone["dlogits"])
    x64, w64 = f64(x), f64(wr)
    # the two calls' logit gradients g and g + dl are each rounded to bf16 and multiplied in
    # float32; dw_router is rounded again, once per split of the tokens (16 at most) and at the end
    h = oracle.backward(host_array(x), host_array(wr), None if b is None else host_array(b), host_array(W1),
                        host_array(W2), k, "bf16", host_array(dy))
    gl = np.abs(h["dlogit"]) * 1.1 + 1e-3 * np.abs(h["dlogit"]).max()  # the layer's own part, from above
    hb = HALF[bf]
    rnd = hb * (2 * gl + np.abs(dl))  # of the two rounded logit gradients
    ref = x64.T @ dl
    mag = np.abs(x64).T @ (gl + np.abs(dl))
    assert_within("dw_router", f64(c["dwr"]) - f64(a["dwr"]), ref,
                  np.abs(x64).T @ rnd + hb * 4 * (np.abs(f64(a["dwr"])) + np.abs(f64(c["dwr"]))) + 2 * hb * mag)
    ref = dl @ w64.T
    both = np.abs(f64(a["dx"])) + np.abs(f64(c["dx"]))
    # dx adds the k expert rows and the router's row, itself rounded to bf16
    assert_within("dx", f64(c["dx"]) - f64(a["dx"]), ref,
                  rnd @ np.abs(w64).T + hb * both + hb * 2 * ((gl + np.abs(dl)) @ np.abs(w64).T))
    assert_within("dbias", f64(c["db"]) - f64(a["db"]), dl.sum(axis=0),
                  (T + 300) * U32 * (2 * gl + np.abs(dl)).sum(axis=0) + 1e-30)
