"""No entropy below 0 and no log probability above 0, however peaked a row is."""
import pytest
import torch

from _helpers import have_gpu
from test_gpu_score import DEV, TYPES, dense  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(3000, 700), (64, 9600)])
def test_signs(dense, dtype, T, V):  # noqa: F811
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, V), generator=g) * 0.2 - 40
    j = torch.randint(0, V, (T,), generator=g)
    x[torch.arange(T), j] = torch.rand(T, generator=g) * 8               # the only one with weight
    x[torch.arange(T), (j + V // 2) % V] = -16 - torch.rand(T, generator=g)
    ids = torch.stack([j, (j + 1) % V], 1).to(torch.int32)
    for scale in (1.0, 1.7, 5.0):
        s = dense.token_logprobs(x.to(dtype).to(DEV), ids.to(DEV), k=3, scale=scale)
        assert (s.entropy >= 0).all() and (s.logprob <= 0).all() and (s.top_logprob <= 0).all()
