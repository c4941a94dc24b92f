"""Token log probabilities under scales from fp32's smallest numbers on, and of logits whose distance passes fp32's range, against the
float64 oracle.  Bounds as in test_gpu_score: a term's exponent is a difference (e of it) times c (2 e) rounded (e), 4 e of |t| in all,
and |t| 2^t < 0.54 for each; scales below 2^-126 have fewer bits, so c's own error is their half step relative."""
import math

import pytest
import torch

from _helpers import have_gpu
from oracle import dense_oracle as D
from test_gpu_score import DEV, E, check, dense, draw  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
WIDE = [torch.bfloat16, torch.float32]
FORMS = [(2, 9600), (800, 700)]                 # a row's CTAs of a cluster, one CTA


def as_f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("scale", [1e-36, 1e-37, 5e-38, 1e-38])
@pytest.mark.parametrize("T,V", FORMS)
@pytest.mark.parametrize("size", [1e9, 1e30, 1e37, 1.5e38])
def test_masked_logits_have_no_weight_under_any_scale(dense, dtype, scale, T, V, size):  # noqa: F811
    scale = as_f32(scale)
    x, ids = draw(T, V, dtype, spread=1.0)
    x = (x.clamp(-2, 2) * size).to(dtype)
    x[:, 1::3] = -math.inf
    x[0, 4:] = -math.inf
    ids[0, 0], ids[T - 1, 0] = 1, 3
    few = [0, 1, T - 1]
    check(dense, x[few], ids[few], 6, scale)
    s = check(dense, x, ids, 6, scale) if T < 10 else dense.token_logprobs(x.to(DEV), ids.to(DEV), k=6, scale=scale)
    assert s.logprob[0, 0] == -math.inf and torch.isfinite(s.entropy).all()


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("T,V", FORMS)
def test_subnormal_scales(dense, dtype, T, V):  # noqa: F811
    """Every token that is not masked is as probable as the next."""
    for scale in (1e-40, 1.5e-45):
        x, ids = draw(T, V, dtype)
        x[:, 1::2] = -math.inf
        s = dense.token_logprobs(x.to(DEV), ids.to(DEV), scale=scale)
        ref = torch.where(ids % 2 == 1, -math.inf, -math.log((V + 1) // 2)).double()
        bound = (V / 256 + 60) * E * (1 + math.log(V))
        got = s.logprob.double().cpu()
        assert torch.equal(torch.isinf(got), torch.isinf(ref)) and ((got - ref).abs()[torch.isfinite(ref)] <= bound).all()
        assert ((s.entropy.double().cpu() - math.log((V + 1) // 2)).abs() <= bound).all()


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("T,V", FORMS)
@pytest.mark.parametrize("scale", [1.0, 0.3, 1e-3, 1e-20, 1e-37, 1e-38])
def test_logits_further_apart_than_fp32_reaches(dense, dtype, T, V, scale):  # noqa: F811
    """Differences past the largest fp32 number, whose product with the scale is a log probability all the same."""
    scale, low = as_f32(scale), torch.finfo(dtype).min
    x, ids = draw(T, V, dtype)
    x[0, :] = low
    x[0, V // 2] = -low
    x[1, 5::7], x[1, 3::7] = 0.75 * -low, 0.7 * low
    ids[0], ids[1] = torch.tensor([0, V // 2, V - 1]), torch.tensor([5, 3, 4])
    check(dense, x[:2], ids[:2], 5, scale)
    if T > 2:
        s = dense.token_logprobs(x.to(DEV), ids.to(DEV), k=5, scale=scale)
        few = torch.tensor([0, 1])
        lp = D.token_logprobs(x[few], ids[few], 5, scale)
        assert torch.equal(s.top_ids[:2].cpu(), lp[3]) and torch.equal(torch.isinf(s.logprob[:2].cpu()), lp[0].abs() > 3.5e38)
