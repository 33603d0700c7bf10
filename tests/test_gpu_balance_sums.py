"""The balance loss over many rows: the means' error does not grow with the batch."""

import pytest
import torch

from gpu_helpers import U32, announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

CASES = [  # T, E: 128 or 256 rows for every thread of a whole launch, by one lane to a whole wave per token
    (1 << 25, 3), (1 << 22, 17), (1 << 20, 100), (1 << 20, 130), (1 << 19, 252),
]


@pytest.mark.parametrize("masked", [False, True], ids=["all", "masked"])
@pytest.mark.parametrize("T,E", CASES)
def test_equal_rows(moe, T, E, masked):
    """Equal logits: every probability is the float32 nearest to 1 / E, so the error of
    each addition has the same sign as the one before for many rows on end.
    mean_prob is off by the rounding of 1 / E, of a workgroup's sum and of the result,
    half a unit each; the loss, coef sum f E mean_prob with sum f = 1, by one more."""
    announce(f"balance equal rows T={T} E={E} masked={masked}")
    p = moe.make_problem(T, 64, E, 1, 64, torch.float32)
    logits = torch.full((T, E), 0.75, device="cuda")
    t = torch.arange(T, device="cuda")
    idx = (t * t % E).to(torch.int32).reshape(T, 1)
    mask = (t % 3 != 1) if masked else None
    loss, mean = torch.empty(1, device="cuda"), torch.empty(E, device="cuda")
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_BALANCE), dtype=torch.uint8, device="cuda")
    moe.moex_balance_loss(p, logits, idx, mask, 2.0, loss, counts, mean, None, ws)
    torch.cuda.synchronize()
    sel = idx.reshape(-1).long() if mask is None else idx.reshape(-1).long()[mask]
    assert torch.equal(counts.long(), torch.bincount(sel, minlength=E))
    assert bool(((mean.double() * E - 1).abs() <= 3.01 * U32).all()), (mean.double() * E - 1).abs().max() / U32
    assert abs(float(loss) / 2.0 - 1) <= 4.01 * U32
