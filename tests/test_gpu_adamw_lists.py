"""Everything that a step of a list in several launches writes, of every tensor, against float64."""

import numpy as np
import pytest
import torch

from ext_helpers import assert_within
from gpu_helpers import U32, announce, f64, needs_gpu
from oracle import train_ops as to
from test_gpu_adamw import B1, B2, BF, EPS, F32, LR, Mirror, params_of

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("clip", [None, float("inf"), 0.25])
@pytest.mark.parametrize("count", [48, 49, 130])
def test_all_of_a_list(moe, count, clip):
    """48 tensors are one launch of the step, 128 one of the norm. Moments and codes bit for bit, as in a short list."""
    announce(f"adamw {count} tensors, all outputs, max_norm={clip}")
    params, grads = params_of([(1 + 61 * i % 5003, BF if i % 3 else F32, BF if i % 2 else F32) for i in range(count)], 61)
    bits = [8 if i % 2 else 32 for i in range(count)]
    factor, decay = [0.5 + i % 4 for i in range(count)], [0.1 * (i % 3) for i in range(count)]
    opt = moe.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decay, lr_factor=factor, bits=bits, max_norm=clip, seed=7)
    ref = Mirror(opt)
    for t in (1, 2):
        ref.before()
        opt.step(grads)
        torch.cuda.synchronize()
        scale = 1.0 if clip is None else float(opt.scale)
        if clip is not None:
            total = np.sqrt(sum(np.sum(f64(g) ** 2) for g in grads))
            assert abs(float(opt.norm) - total) <= 2 * U32 * total
            want = min(1.0, clip / total)
            assert abs(scale - want) <= 2 * U32 * want and (scale == 1.0) == (clip >= total)
        assert opt.counter.tolist() == [t, 0]
        for i in range(count):
            g = f64(grads[i]) * np.float64(scale)
            m = B1 * ref.m[i] + (1 - B1) * g
            v = B2 * ref.v[i] + ((1 - B2) * g) * g
            p = to.adamw(ref.p[i], g, ref.m[i], ref.v[i], t, LR * factor[i], B1, B2, EPS, decay[i])[0]
            got = f64(params[i] if opt.master[i] is None else opt.master[i])
            assert_within(f"param {i}", got, p, 2.0 ** -20 * np.abs(p - ref.p[i]) + 2 * U32 * (np.abs(p) + np.abs(ref.p[i])))
            if opt.master[i] is not None:
                assert torch.equal(params[i], opt.master[i].to(BF).view_as(params[i])), i
            if bits[i] == 32:
                assert np.array_equal(opt.m[i].cpu().numpy(), m.astype(np.float32)), i
                assert np.array_equal(opt.v[i].cpu().numpy(), v.astype(np.float32)), i
                continue
            r = to.draws(g.size, 7, t, i)
            for name, x, rr, c, s, tab in (("m", m, r & 0xFFFF, opt.m[i], opt.m_scale[i], to.E4M3_POS),
                                           ("v", v, r >> 16, opt.v[i], opt.v_scale[i], to.E5M2_POS)):
                codes, e = to.round_stochastic(x, rr, tab, name == "v")
                assert np.array_equal(s.cpu().numpy().astype(np.int64) - 127, e), (name, i)
                assert np.array_equal(c.view(torch.uint8).cpu().numpy(), codes), (name, i)
