"""Index arrays of tokens that name experts more than once, in one block of 256 tokens and in
several, against a sort; and the time of the most repetitive ones."""

import numpy as np
import pytest
import torch

from ext_helpers import gen
from gpu_helpers import announce, i64, needs_gpu
from oracle import train_ops as to
from test_gpu_canary import Guarded

pytestmark = [pytest.mark.gpu, needs_gpu]

I32 = torch.int32


class Index:
    """moet_dispatch of 64-wide rows, all outputs guarded."""

    def __init__(self, moe, idx, E):
        self.moe, self.idx, self.E = moe, idx.to(I32).contiguous(), E
        self.T, self.k = T, k = idx.shape
        self.p = moe.make_problem(T, 64, E, k, 64, torch.float32)
        self.x = torch.randn((T, 64), generator=gen(1), device="cuda")
        shapes = {"counts": (E,), "offsets": (E + 1,), "perm": (T * k,), "inv": (T * k,)}
        self.out = {n: Guarded(s, I32) for n, s in shapes.items()}
        self.out["x_perm"] = Guarded((T * k, 64), torch.float32)
        self.out["ws"] = Guarded((moe.moet_workspace_size(self.p, moe.MOET_STAGE_DISPATCH),), torch.uint8)

    def run(self):
        self.moe.moet_dispatch(self.p, self.idx, None, self.x, *(self.out[n].t for n in ("counts", "offsets", "perm", "inv", "x_perm", "ws")))

    def check(self):
        for n in ("perm", "x_perm"):
            self.out[n].t.zero_()
        self.run()
        torch.cuda.synchronize()
        ref = to.dispatch_index(i64(self.idx), self.E)
        n = ref["perm"].size
        for name in ("counts", "offsets", "inv"):
            assert np.array_equal(i64(self.out[name].t), ref[name]), name
        perm = i64(self.out["perm"].t)
        assert np.array_equal(perm[:n], ref["perm"]) and not perm[n:].any()
        assert torch.equal(self.out["x_perm"].t[:n], self.x[torch.from_numpy(ref["perm"]).cuda()])
        assert not self.out["x_perm"].t[n:].any() and all(g.intact() for g in self.out.values())


@pytest.mark.parametrize("T,k,E", [(T, k, E) for T, k in ((1200, 8), (1500, 3), (257 * 8, 1), (1025, 17), (17000, 4))
                                   for E in (1, 2, 31, 32, 33, 64, 65, 256) if k <= E])
def test_random_repeats(moe, T, k, E):
    announce(f"repeats T={T} k={k} E={E}")
    idx = torch.randint(0, E, (T, k), generator=gen(T + E), device="cuda")
    gone = torch.rand((T, k), generator=gen(2), device="cuda")
    idx = torch.where(gone < 0.05, -1, torch.where(gone < 0.1, E, idx))
    idx.view(-1)[::301] = -2 ** 31  # far outside
    idx.view(-1)[7::307] = 2 ** 31 - 1
    Index(moe, idx, E).check()


@pytest.mark.parametrize("T,k,E", [(1100, 200, 200), (600, 256, 256), (1025, 40, 40)])
@pytest.mark.parametrize("who", ["all", "one token", "every third", "two in turn", "all but the last"])
def test_one_expert_throughout(moe, T, k, E, who):
    """Tokens that name one expert with every selection, beside tokens that name each once, over several blocks."""
    announce(f"repeats {who} T={T} k={k} E={E}")
    idx = torch.rand((T, E), generator=gen(3), device="cuda").argsort(1)[:, :k].contiguous()
    e = E - 1
    if who == "all":
        idx.fill_(e)
    elif who == "one token":
        idx[300] = e
    elif who == "every third":
        idx[::3] = e
    elif who == "two in turn":
        idx[:, 0::2], idx[:, 1::2] = 0, e
    else:
        idx[:, :k - 1] = e
        idx[:, k - 1] = 5
    Index(moe, idx, E).check()


def test_first_of_a_block_alone(moe):
    """Blocks without repeats beside one that has them: both ways of ranking in one launch."""
    announce("repeats in one block of five")
    idx = torch.rand((1280, 64), generator=gen(4), device="cuda").argsort(1)[:, :8].contiguous()
    idx[512:520] = 9
    Index(moe, idx, 64).check()


def test_cost_is_linear_in_the_selections(moe):
    """2048 tokens that name one of 256 experts 256 times each: milliseconds at most, where ranks that count a
    token's earlier selections for each of 256 levels read some eight million selections a thread."""
    announce("time of 256 repeats a token")
    c = Index(moe, torch.full((2048, 256), 7, device="cuda"), 256)
    c.run()
    torch.cuda.synchronize()
    best = 1e9
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        c.run()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    assert best < 20.0, best
    c.check()
