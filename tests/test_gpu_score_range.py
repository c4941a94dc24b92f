"""Token log probabilities of logits of any finite size, against the float64 oracle: rows far from 0, where the product of a logit and
the scale has rounding errors of whole units, and rows masked by a finite value.  The bounds are those of test_gpu_score; where a
row's logits are equal every term is 2^0 and only the sum (n roundings, relative) and its logarithm (2 e of it) are off."""
import math

import pytest
import torch

from _helpers import have_gpu
from oracle import dense_oracle as D
from test_gpu_score import DEV, E, check, dense, draw  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
WIDE = [torch.bfloat16, torch.float32]          # f16 ends at 65504
SIZES = [1e9, 2e9, 1e10, -1e9, -1e10, 1e12, 1e20, -1e20, 1e30, -1e30, 2.0 ** 24, -2.0 ** 25]
FORMS = [(2, 9600), (800, 700)]                 # a row's CTAs of a cluster, one CTA


def n_sum(V):
    return V / 256 + 56


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("scale", [1.0, 30.0])
@pytest.mark.parametrize("T,V", FORMS)
def test_equal_logits_of_any_size(dense, dtype, scale, T, V):  # noqa: F811
    """ln V is the entropy and -ln V every log probability, wherever the logits lie."""
    for first in range(0, len(SIZES), T):
        sizes = SIZES[first:first + T]
        x, ids = draw(T, V, dtype)
        for t, size in enumerate(sizes):
            x[t] = size
        few = list(range(len(sizes)))
        s = dense.token_logprobs(x.to(DEV), ids.to(DEV), k=5, scale=scale)
        bound = (n_sum(V) + 4) * E * (1 + math.log(V))
        for got, ref in ((s.logprob, -math.log(V)), (s.top_logprob, -math.log(V)), (s.entropy, math.log(V))):
            assert ((got[few].double().cpu() - ref).abs() <= bound).all()
        assert s.top_ids[few].tolist() == [list(range(5))] * len(few)
        lse = x[few, 0].double() * scale + math.log(V)
        assert ((s.lse[few].double().cpu() - lse).abs() <= bound + 2 * E * lse.abs()).all()
        if T > len(SIZES):
            check(dense, x[[0, T - 1]], ids[[0, T - 1]], 5, scale)
            assert torch.isfinite(s.lse).all() and torch.isfinite(s.logprob).all() and torch.isfinite(s.entropy).all()


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("scale", [1.0, 30.0])
@pytest.mark.parametrize("T,V", FORMS)
def test_one_large_logit_among_ordinary_ones(dense, dtype, scale, T, V):  # noqa: F811
    for size in SIZES:
        x, ids = draw(T, V, dtype)
        x[0, V // 3], x[T - 1, V - 1], x[T - 1, 0] = size, size, size
        ids[0, 0] = V // 3
        few = [0, T - 1]
        check(dense, x[few], ids[few], 4, scale)
        s = dense.token_logprobs(x.to(DEV), ids.to(DEV), k=4, scale=scale)
        if size > 0:
            assert s.logprob[0, 0] == 0 and abs(float(s.entropy[0])) <= 20 * E
            assert abs(float(s.top_logprob[T - 1, 1]) + math.log(2)) <= 20 * E


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("scale", [1.0, 30.0])
@pytest.mark.parametrize("T,V", FORMS)
@pytest.mark.parametrize("mask", [-1e9, -1e10, -1e30])
@pytest.mark.parametrize("keep", [2, 50, 3001])
def test_rows_masked_by_a_finite_value(dense, dtype, scale, T, V, mask, keep):  # noqa: F811
    """One token in `keep` is not masked (in rows of 700 at the largest, one): masked ones have no weight, so the row is that of the
    others alone."""
    x, ids = draw(T, V, dtype, spread=2.5 / scale)
    j = torch.arange(V)
    there = j % min(keep, V) == 1
    bare = torch.where(there, x, torch.full((), -math.inf, dtype=dtype))
    x = torch.where(there, x, torch.full((), mask, dtype=dtype))
    ids = j[there][torch.arange(T)[:, None] % int(there.sum())].to(torch.int32)
    s = dense.token_logprobs(x.to(DEV), ids.to(DEV), k=3, scale=scale)
    few = [0, 1, T - 1]
    lp, h, lse, top, toplp = D.token_logprobs(bare[few], ids[few], min(3, int(there.sum())), scale)
    big = float((bare[few].double() * scale).abs()[torch.isfinite(bare[few])].max())
    bound = E * (6 + n_sum(V) + 8 * big)
    assert ((s.logprob[few].double().cpu() - lp).abs() <= bound).all() and ((s.lse[few].double().cpu() - lse).abs() <= bound).all()
    assert ((s.entropy[few].double().cpu() - h).abs() <= bound + E * ((n_sum(V) + 16) * (1 + h) + 512)).all()
    assert torch.equal(s.top_ids[few, :top.shape[1]].cpu(), top)
    assert ((s.top_logprob[few, :top.shape[1]].double().cpu() - toplp).abs() <= bound).all()


@pytest.mark.parametrize("dtype", WIDE)
def test_a_part_of_a_long_row_all_masked(dense, dtype):  # noqa: F811
    """Whole warps and CTAs that see nothing but the mask's value beside those that see ordinary logits."""
    x, ids = draw(3, 131072, dtype)
    x[0, 20000:] = -1e10
    x[1, :100000] = -1e30
    x[2, 8 * 1024:] = -1e10
    bare = torch.where(x < -1e8, torch.full((), -math.inf, dtype=dtype), x)
    s = dense.token_logprobs(x.to(DEV), None, k=8)
    _, h, lse, top, toplp = D.token_logprobs(bare, None, 8)
    bound = E * (6 + n_sum(131072) + 8 * 15)
    assert ((s.lse.double().cpu() - lse).abs() <= bound).all() and torch.equal(s.top_ids.cpu(), top)
    assert ((s.top_logprob.double().cpu() - toplp).abs() <= bound).all()
    assert ((s.entropy.double().cpu() - h).abs() <= bound + E * ((n_sum(131072) + 16) * (1 + h) + 512)).all()
