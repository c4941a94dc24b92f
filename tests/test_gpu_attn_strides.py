"""The stride of a dimension of one is open: torch may give it any value, and no call depends on it."""
import pytest
import torch

from _helpers import have_gpu
from test_gpu_kv import DEV, attn, i32, make, same  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]


def open_strides(x, odd=5):
    """x with an odd stride in every dimension of one."""
    return x.as_strided(x.shape, [odd if n == 1 else s for n, s in zip(x.shape, x.stride())])


@pytest.mark.parametrize("T,H", [(7, 1), (1, 3), (1, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope(attn, T, H, dtype):  # noqa: F811
    x = torch.randn((T, H, 64), generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    pos, tab = i32(list(range(T))), attn.rope_table(16, 64, device=DEV)
    want = attn.rope(x, pos, tab)
    assert torch.equal(attn.rope(open_strides(x), pos, tab), want)
    out = open_strides(torch.zeros_like(x))
    assert torch.equal(attn.rope(x, pos, tab, out=out), want)
    y = open_strides(x.clone())
    assert torch.equal(attn.rope(y, pos, tab, out=y), want)


@pytest.mark.parametrize("layers,T,H,qh", [(1, 5, 1, 1), (1, 5, 1, 4), (2, 1, 1, 1), (1, 1, 2, 2)])
def test_append(attn, layers, T, H, qh):  # noqa: F811
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn((layers, T, H, 16), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn((T, qh, 16), generator=g).to(torch.bfloat16).to(DEV)
    cu, pos, tab = i32([0, T]), i32(list(range(T))), attn.rope_table(16, 16, device=DEV)
    got = []
    for f in (lambda x: x, open_strides):
        cache, _ = make(attn, layers=layers, H=H)
        start = cache.extend(i32([0]), i32([2 * T]))
        cache.append(f(k), f(v), cu, i32([0]), start, layer=None)
        qo = cache.append(f(k[0]), f(v[0]), cu, i32([0]), start + T, layer=0, q=f(q), pos=pos, cos_sin=tab)
        got.append((cache.pool, qo))
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])
