"""Scores that are not finite: out and lse by the formulas (out = sum exp(s) v / sum exp(s), lse = ln sum exp(s))."""
import math

import pytest
import torch

from _helpers import have_gpu
from test_gpu_attention import B16, DEV, H16, Case, attn  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("dtype,Hq,Hk,D,ps,new,ctx", [(B16, 4, 2, 64, 16, [6], [300]),            # whole, both streams merged
                                                      (H16, 4, 1, 128, 32, [5], [9000]),           # pieces joined
                                                      (H16, 2, 2, 64, 64, [700], [200]),           # two row tiles
                                                      (B16, 4, 1, 128, 16, [300, 400], [0, 60])])
@pytest.mark.parametrize("at", [0.0, 0.5, 0.99])
def test_infinite_keys(attn, dtype, Hq, Hk, D, ps, new, ctx, at):  # noqa: F811
    """An infinity in one column of a cached key: a row whose query is positive there has a score of +inf, out is inf / inf and
    lse is +inf; one whose query is negative has -inf, as if it did not see the key."""
    c = Case(attn, dtype, Hq, Hk, D, ps, new, ctx, seed=51)
    sign = torch.where(torch.arange(c.q.shape[0]) % 2 == 0, 1.0, -1.0)
    c.q[:, :, 3] = (c.q[:, :, 3].abs().float() + 0.125).to(dtype) * sign[:, None].to(dtype)
    pos = []
    for b, (m, s) in enumerate(zip(new, ctx)):
        pos.append(int(at * (s + m - 1)))
        c.cache.pool[0, int(c.cache.table[c.slots[b], pos[b] // ps]), 0, :, pos[b] % ps, 3] = math.inf
    out, lse = c.run()
    for b in range(len(new)):
        for i in range(new[b]):
            row = c.cu[b] + i
            if pos[b] > ctx[b] + i:
                continue                                 # not seen
            if row % 2 == 0:
                assert (lse[row] == math.inf).all() and torch.isnan(out[row]).all(), (b, i)
                c.see[b][i] = []                         # checked: out of the comparison below
                out[row], lse[row] = 0, -math.inf
            else:
                c.see[b][i] = [j for j in c.see[b][i] if j != pos[b]]
    c.check(out, lse)


@pytest.mark.parametrize("dtype,Hq,D,new,ctx", [(B16, 2, 64, [3], [500]), (H16, 1, 128, [300], [0])])
def test_nan_beats_infinity(attn, dtype, Hq, D, new, ctx):  # noqa: F811
    c = Case(attn, dtype, Hq, 1, D, 16, new, ctx, seed=52)
    c.q[:, :, 3] = 1.0
    for pos, x in ((20, math.inf), (21, math.nan)):
        c.cache.pool[0, int(c.cache.table[c.slots[0], pos // 16]), 0, :, pos % 16, 3] = x
    out, lse = c.run()
    first = max(0, 21 - ctx[0])
    assert torch.isnan(out[first:]).all() and torch.isnan(lse[first:]).all()


def test_several_infinite_keys(attn):  # noqa: F811
    c = Case(attn, B16, 2, 1, 64, 16, [4], [3000], seed=53)
    c.q[:, :, 3] = 1.0
    for pos in (5, 6, 700, 1500, 2999):
        c.cache.pool[0, int(c.cache.table[c.slots[0], pos // 16]), 0, :, pos % 16, 3] = math.inf
    out, lse = c.run()
    assert torch.isnan(out).all() and (lse == math.inf).all()
