"""New tokens whose values are not finite: what they cost, and which rows they reach, over many tiles, items and heads.

Expectations are exact.  A row's softmax does not look at V, so the columns without a bad value keep their bits; in the others
a row that sees bad values has their sum (an infinity or NaN) and the others keep theirs."""
import math
import random

import pytest
import torch

from _helpers import have_gpu
from test_gpu_attention import B16, DEV, H16, Case, attn, i32  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]


def plant(c, bads):
    """bads: (sequence, new token, K/V head, column, value)."""
    ps = c.cache.pool.shape[4]
    for b, at, h, d, x in bads:
        pos = c.ctx[b] + at
        c.cache.pool[0, int(c.cache.table[c.slots[b], pos // ps]), 1, h, pos % ps, d] = x


def expected(c, clean, bads, sees=None):
    """sees[b](token) -> bool per row of sequence b; None: causal."""
    want, grp = clean.clone(), clean.shape[1] // c.Hk
    for b, at, h, d, x in bads:
        rows = torch.arange(c.new[b], device=DEV)
        hit = rows >= at if sees is None else sees[b](at)
        rows = rows[hit] + c.cu[b]
        want[rows, h * grp:(h + 1) * grp, d] += x
    return want


def same(out, want):
    return torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out.nan_to_num(0.0, 1e4, -1e4),
                                                                            want.nan_to_num(0.0, 1e4, -1e4))


def some(r, c, per):
    return [(b, at, r.randrange(c.Hk), r.randrange(c.D), r.choice([math.inf, -math.inf, math.nan]))
            for b in range(len(c.new)) if c.new[b] for at in r.sample(range(c.new[b]), min(per, c.new[b]))]


@pytest.mark.parametrize("dtype,Hq,Hk,D,ps,new,ctx", [
    (B16, 8, 2, 128, 64, [3001, 1, 200], [70, 500, 0]),          # both row tiles of an item in one key tile
    (H16, 3, 3, 64, 16, [2900], [37]),                           # row tiles a key tile apart
    (B16, 6, 2, 72, 32, [1500, 333], [0, 1000]),                 # groups that do not divide a tile of rows
    (H16, 16, 2, 128, 256, [40, 9, 120, 0, 1], [2000, 100, 5, 9, 3000]),   # one row tile an item, split along the keys
    (B16, 1, 1, 40, 8, [100, 128, 3], [1, 127, 129])])
@pytest.mark.parametrize("per", [1, 40])
def test_only_the_rows_that_see_them(attn, dtype, Hq, Hk, D, ps, new, ctx, per):  # noqa: F811
    c = Case(attn, dtype, Hq, Hk, D, ps, new, ctx, seed=31)
    clean, lse0 = c.run()
    bads = some(random.Random(per), c, per)
    plant(c, bads)
    want = expected(c, clean, bads)
    first = None
    for _ in range(2):
        out, lse = c.run()
        assert torch.equal(lse, lse0) and same(out, want)
        first = out if first is None else first
        assert torch.equal(first.view(torch.int16), out.view(torch.int16)), "runs agree"


@pytest.mark.parametrize("dtype,Hq,Hk,D,new,ctx", [(B16, 2, 1, 64, [8500], [100]),                  # two row tiles an item
                                                   (H16, 1, 1, 128, [8400] + [1] * 70, [55] * 71)])  # one
def test_masks_over_more_tiles_than_are_noted_apart(attn, dtype, Hq, Hk, D, new, ctx):  # noqa: F811
    c = Case(attn, dtype, Hq, Hk, D, 128, new, ctx, seed=32)
    words = -(-max(new) // 32) - 3                   # the last tokens are visible to no row
    g = torch.Generator().manual_seed(5)
    mask = torch.randint(-2 ** 31, 2 ** 31, (sum(new), words), generator=g).to(torch.int32).to(DEV)
    mask[7] = 0                                      # padding
    c.mask = mask
    clean, lse0 = c.run()
    bads = some(random.Random(9), c, 30) + [(0, new[0] - 1, 0, 3, math.nan), (0, 64, 0, 5, math.inf), (0, 64 + 8192, 0, 6, math.inf)]
    plant(c, bads)

    def sees(b):
        rows = mask[c.cu[b]:c.cu[b + 1]]
        return lambda at: (rows[:, at // 32] >> (at % 32) & 1).bool() if at < 32 * words else torch.zeros(c.new[b], dtype=torch.bool,
                                                                                                         device=DEV)
    want = expected(c, clean, bads, [sees(b) for b in range(len(new))])
    out, lse = c.run()
    assert torch.equal(lse, lse0) and same(out, want)
    assert not out[7].any()


def test_every_value_bad(attn):  # noqa: F811
    c = Case(attn, B16, 4, 2, 64, 64, [700, 30], [0, 300], seed=33)
    _, lse0 = c.run()
    for b in range(2):
        plant(c, [(b, at, slice(None), slice(None), math.nan) for at in range(c.new[b])])
    out, lse = c.run()
    assert torch.isnan(out).all() and torch.equal(lse, lse0)


def timed(c):
    q, cu, seqs, start = c.q.to(DEV), i32(c.cu), i32(c.slots), i32(c.ctx)
    best = math.inf
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        c.attn.attention(q, c.cache, cu, seqs, start, mask=c.mask)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("Hq,Hk,D,new,ctx", [(8, 8, 128, [8191], [0]), (8, 2, 64, [60, 3, 33], [20000, 9000, 15000])])
def test_the_cost_is_that_of_the_bad_tokens(attn, Hq, Hk, D, new, ctx):  # noqa: F811
    """A bad value of one head and token costs the items it lies in a look at one token: not every later item a walk over all
    its new tokens (8191 tokens of 128 values, one after the other, would take tens of milliseconds)."""
    c = Case(attn, B16, Hq, Hk, D, 64, new, ctx, seed=34)
    clean = timed(c)
    plant(c, [(0, 5, 0, 3, math.inf), (0, new[0] // 2, 1, 0, math.nan)])
    few = timed(c)
    assert few < 1.5 * clean + 0.1, (clean, few)
    plant(c, [(0, at, slice(None), slice(None), math.inf) for at in range(new[0] // 3, new[0] // 3 + 16)])
    many = timed(c)
    assert many < 2 * clean + 0.5, (clean, many)
    print(f"attention {clean * 1e3:.0f} us, two bad values {few * 1e3:.0f} us, 16 bad tokens {many * 1e3:.0f} us")
