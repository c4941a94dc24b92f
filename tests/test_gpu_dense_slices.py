"""Slices of ids, scales, biases and weights that start on any element, as they come out of a prompt's tokens, a batch's rows and a
fused projection's channels."""
import pytest
import torch

from _helpers import have_gpu
from test_gpu_linear8 import DEV, draw

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def dense():
    from weight_only_int4_route_gb300 import build, dense, moe
    build.build()
    moe.lib()
    return dense


@pytest.mark.parametrize("first", [1, 2, 3, 5])
def test_slices_at_every_offset(dense, first):
    a, sa, w, sw, b = (t.to(DEV) for t in draw(40, 150, 192))
    whole = dense.linear_w8a8(a, sa, w, sw, b, out_dtype=torch.float32)
    for rows in (3, 30):
        part = slice(first, first + rows)
        assert torch.equal(dense.linear_w8a8(a[part], sa[part], w, sw, b, out_dtype=torch.float32), whole[part])
        channels = slice(first, first + 64)
        assert torch.equal(dense.linear_w8a8(a[part], sa[part], w[channels], sw[channels], b[channels], out_dtype=torch.float32),
                           whole[part, channels])
    tokens = torch.randint(0, 150, (41,), dtype=torch.int32, device=DEV)
    s = dense.token_logprobs(whole, tokens[1:], k=3)
    assert torch.equal(dense.token_logprobs(whole[first:], tokens[1 + first:], k=3).logprob, s.logprob[first:])
    assert torch.equal(s.logprob, dense.token_logprobs(whole, tokens[1:].clone()).logprob)
    gain = torch.rand(600, device=DEV).half()
    x = torch.randn((7, 192), device=DEV).half()
    assert torch.equal(dense.rmsnorm(x, gain[first:first + 192]).y, dense.rmsnorm(x, gain[first:first + 192].clone()).y)


def test_slices_captured_and_replayed(dense):
    a, sa, w, sw, b = (t.to(DEV) for t in draw(40, 150, 192))
    tokens = torch.randint(0, 150, (41,), dtype=torch.int32, device=DEV)
    step = lambda: dense.token_logprobs(dense.linear_w8a8(a[1:], sa[1:], w, sw, b, out_dtype=torch.float32), tokens[2:], k=2)  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        tokens.copy_(torch.roll(tokens, 1))
        sa.mul_(1.25)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(held, step()))
