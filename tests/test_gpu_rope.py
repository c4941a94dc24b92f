"""Rotary positions on the GPU against the float64 oracle.

Bounds.  A turned element is a c -+ b s: two products and a sum in fp32 (three roundings, 2^-24 each, of terms at most
|a| + |b|), then one rounding to the output type (u = 2^-8 bf16, 2^-11 f16, 2^-24 f32 of the result): the
bound below takes four fp32 roundings.  A table entry is a 64-bit value rounded to fp32 once (2^-25 relative to 1, plus
the 64-bit angle's own error, below 2^-30 for positions up to 2^20); the bound is 2^-23."""
import pytest
import torch

from _helpers import have_gpu
from oracle import attn_oracle as A

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def attn():
    from weight_only_int4_route_gb300 import attn, build, moe
    build.build()
    moe.lib()
    return attn


def check(got, x, pos, tab, inter, inverse):
    ref = A.rope(x, pos, tab, inter, inverse)
    rot = tab.shape[1]
    assert torch.equal(got[..., rot:].cpu(), x[..., rot:]), "the unturned part is copied"
    big = x.double().abs().amax(-1, keepdim=True) * 2 * max(1.0, float(tab.abs().max()))
    bound = U[x.dtype] * ref.abs() + 4 * 2.0 ** -24 * big
    bad = (got.double().cpu() - ref).abs() > bound
    assert not bad.any(), float(((got.double().cpu() - ref).abs() / bound).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,D,rot,inter,inverse", [
    (1, 1, 8, 2, False, False), (1, 32, 128, 128, False, False), (7, 3, 64, 64, True, True), (33, 5, 96, 48, False, True),
    (9, 2, 80, 40, False, False), (9, 2, 80, 40, True, False), (5, 4, 128, 16, False, True), (6, 2, 24, 12, False, False),
    (6, 2, 24, 6, True, True), (300, 2, 64, 20, False, False), (4, 1, 256, 256, True, False), (130, 17, 64, 64, False, True)])
def test_rope(attn, dtype, T, H, D, rot, inter, inverse):
    g = torch.Generator().manual_seed(T * 1000 + D)
    x = torch.randn((T, H, D), generator=g).to(dtype)
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32)
    tab = A.rope_table(range(500), rot).float()
    out = attn.rope(x.to(DEV), pos.to(DEV), tab.to(DEV), interleaved=inter, inverse=inverse)
    check(out, x, pos, tab.double(), inter, inverse)


@pytest.mark.parametrize("inter", [False, True])
def test_strides_and_in_place(attn, inter):
    """A slice of a fused projection (token stride), heads apart (head stride), and in place; neighbours stay as they were."""
    g = torch.Generator().manual_seed(3)
    T, H, D = 21, 6, 64
    whole = torch.randn((T, 3 * H * D), generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 99, (T,), generator=g, dtype=torch.int32)
    tab = A.rope_table(range(99), 32).float()
    w = whole.to(DEV)
    x = w[:, H * D:2 * H * D].unflatten(1, (H, D))
    ref = attn.rope(x.contiguous(), pos.to(DEV), tab.to(DEV), interleaved=inter)
    assert torch.equal(attn.rope(x, pos.to(DEV), tab.to(DEV), interleaved=inter), ref)
    spaced = torch.zeros((T, 2 * H, D), dtype=x.dtype, device=DEV)
    attn.rope(x, pos.to(DEV), tab.to(DEV), interleaved=inter, out=spaced[:, ::2])
    assert torch.equal(spaced[:, ::2], ref) and not spaced[:, 1::2].any()
    check(ref, whole[:, H * D:2 * H * D].unflatten(1, (H, D)), pos, tab.double(), inter, False)
    attn.rope(x, pos.to(DEV), tab.to(DEV), interleaved=inter, out=x)
    assert torch.equal(x, ref)
    assert torch.equal(w[:, :H * D].cpu(), whole[:, :H * D]) and torch.equal(w[:, 2 * H * D:].cpu(), whole[:, 2 * H * D:])


def test_positions_outside_the_table(attn):
    x = torch.randn((5, 2, 16), generator=torch.Generator().manual_seed(4))
    pos = torch.tensor([0, -1, 7, 8, 2 ** 31 - 1], dtype=torch.int32)
    tab = A.rope_table(range(8), 8).float()
    out = attn.rope(x.to(DEV), pos.to(DEV), tab.to(DEV)).cpu()
    assert torch.isfinite(out[[0, 2]]).all()
    assert torch.isnan(out[[1, 3, 4], :, :8]).all() and torch.equal(out[..., 8:], x[..., 8:])


def test_nan_and_infinity_stay_in_their_pair(attn):
    x = torch.ones((1, 1, 16))
    x[0, 0, 1], x[0, 0, 2] = float("nan"), float("inf")
    out = attn.rope(x.to(DEV), torch.tensor([3], dtype=torch.int32, device=DEV), A.rope_table(range(8), 16).float().to(DEV)).cpu()
    bad = ~torch.isfinite(out[0, 0])
    assert bad.nonzero().flatten().tolist() == [1, 2, 9, 10]


def test_gradient_by_differences(attn):
    """The inverse is the gradient of <w, rope(x)>: the map is linear, so a difference of step 1 has no truncation
    error; each of the D terms rounds three times."""
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn((1, 1, 32), generator=g), torch.randn((1, 1, 32), generator=g)
    pos = torch.tensor([77], dtype=torch.int32, device=DEV)
    tab = A.rope_table(range(99), 32).float().to(DEV)
    grad = attn.rope(w.to(DEV), pos, tab, inverse=True).cpu()
    base = attn.rope(x.to(DEV), pos, tab).cpu().double()
    for d in range(32):
        e = torch.zeros_like(x)
        e[0, 0, d] = 1.0
        diff = ((attn.rope((x + e).to(DEV), pos, tab).cpu().double() - base) * w).sum()
        assert abs(float(diff - grad[0, 0, d])) < 32 * 8 * 2.0 ** -24 * 5 * 5


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0, base=500000.0),
                                dict(scaling="parts", factor=16.0, original=4096)])
@pytest.mark.parametrize("rot", [4, 64, 128])
def test_table(attn, kw, rot):
    n = 1 << 20
    got = attn.rope_table(n, rot, device=DEV, **kw)
    assert got.shape == (n, rot)
    rows = [0, 1, 2, 4095, 4096, 131071, n - 1]
    ref = A.rope_table(rows, rot, **kw)
    assert float((got[rows].double().cpu() - ref).abs().max()) < 2.0 ** -23 * 1.5


def test_large_strides(attn):
    """Offsets past 2^31 elements: the last rows of a tensor of 2^32 bytes and more."""
    T, H, D = 70000, 256, 128            # 2.3e9 elements
    x = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
    x[-2:] = torch.randn((2, H, D), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    x[:1] = 1.0
    pos = torch.full((T,), 5, dtype=torch.int32, device=DEV)
    tab = A.rope_table(range(8), D).float()
    keep = x[-2:].cpu()
    out = attn.rope(x, pos, tab.to(DEV), out=x)
    check(out[-2:], keep, torch.tensor([5, 5]), tab.double(), False, False)
