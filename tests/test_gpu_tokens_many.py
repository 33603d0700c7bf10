"""More tokens than a launch has waves: the rows' kernels go on by strides, and the index's launches
are of many blocks. Values are small whole numbers, so that every product and sum is exact."""

import torch
import pytest

from ext_helpers import gen
from gpu_helpers import announce, needs_gpu
from test_gpu_tokens import BF, F32, I32, new

pytestmark = [pytest.mark.gpu, needs_gpu]


def test_past_the_launchs_waves(moe):
    """2^24 waves are the most of a launch; (1 << 24) + 3001 tokens of one selection and one wave each."""
    T, d, E = (1 << 24) + 3001, 64, 5
    announce(f"tokens T={T} d={d}")
    p = moe.make_problem(T, d, E, 1, 64, BF)
    g = gen(121)
    idx = torch.randint(-1, E, (T, 1), generator=g, device="cuda").to(I32)
    x = torch.randint(-8, 9, (T, d), generator=g, device="cuda", dtype=torch.int8).to(BF)
    w = torch.randint(1, 5, (T, 1), generator=g, device="cuda").float()
    counts, offsets, perm, inv = new((E,), I32), new((E + 1,), I32), new((T,), I32), new((T,), I32)
    x_perm, y, dx, dw = torch.zeros_like(x), new((T, d), BF), new((T, d), BF), new((T, 1), F32)
    ws = new((moe.moet_workspace_size(p, moe.MOET_STAGE_DISPATCH),), torch.uint8)
    moe.moet_dispatch(p, idx, w, x, counts, offsets, perm, inv, x_perm, ws)
    e = idx.view(-1).long()
    live = (e >= 0).nonzero().view(-1)
    order = live[torch.sort(e[live], stable=True).indices]
    n = order.numel()
    assert torch.equal(counts.long(), torch.bincount(e[live], minlength=E)) and int(offsets[E]) == n
    assert torch.equal(perm[:n].long(), order)
    want = torch.full((T,), -1, dtype=torch.long, device="cuda")
    want[order] = torch.arange(n, device="cuda")
    assert torch.equal(inv.long(), want)
    assert torch.equal(x_perm[:n], (x[order].float() * w[order]).to(BF)) and not x_perm[n:].any()
    moe.moet_combine(p, x_perm, inv, None, x, y)
    kept = (e >= 0)[:, None]
    both = x.float() * (1 + w * kept)
    assert torch.equal(y, both.to(BF))
    moe.moet_dispatch_backward(p, x_perm, inv, x, w, None, dx, dw)
    assert torch.equal(dx, (x.float() * w * w * kept).to(BF))
    dots = (x.float() * (x.float() * w)).sum(1, keepdim=True) * kept
    assert torch.equal(dw, dots)
    dy_perm, dg = torch.zeros_like(x), new((T, 1), F32)
    moe.moet_combine_backward(p, x, inv, x_perm, w, dy_perm, dg)
    torch.cuda.synchronize()
    assert torch.equal(dy_perm, x_perm) and torch.equal(dg, dots)
