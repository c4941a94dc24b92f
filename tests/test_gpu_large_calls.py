"""Rotations and cache appends of large calls, where a thread takes several heads: odd head counts, partial rotation, both
layouts, every type, with and without queries.  (Calls are large from 152 x 1024 x 4 vectors on, x 8 without pairs of them.)

The rotation's reference is the formula in 64 bits; its bound is that of small calls: four fp32 roundings (2^-24 each) of terms
of at most |a| + |b|, and one rounding to the type of the result (u)."""
import pytest
import torch

from _helpers import have_gpu
from test_gpu_kv import attn, i32  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
DEV = "cuda:0"
B16, H16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {B16: 2.0 ** -8, H16: 2.0 ** -11, F32: 2.0 ** -24}


def vectors(dtype, D, rot, inter, in_place=False):
    """16-byte vectors (or what the rotated pairs allow) of a head that are visited, pairs of them counted once."""
    unit, v = rot if inter else rot // 2, 16 // dtype.itemsize
    while unit % v:
        v //= 2
    return (unit + (0 if in_place else D - rot)) // v


def turned(x, pos, tab, inter, inverse):
    """The formula in 64 bits."""
    rot = tab.shape[1]
    a = tab.double()[pos.long()]
    cos, sin = a[:, None, :rot // 2], a[:, None, rot // 2:] * (-1 if inverse else 1)
    y = x.double().clone()
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    p, q = x[..., lo].double(), x[..., hi].double()
    y[..., lo], y[..., hi] = p * cos - q * sin, p * sin + q * cos
    return y


@pytest.mark.parametrize("dtype,T,H,D,rot,inter,inverse,in_place", [
    (B16, 20001, 7, 128, 64, False, False, False), (B16, 20001, 13, 128, 64, True, False, False),
    (H16, 30011, 5, 96, 96, False, True, True), (H16, 40011, 9, 96, 32, True, True, True),
    (F32, 19001, 3, 128, 128, False, False, False), (F32, 9001, 11, 128, 96, True, True, False),
    (F32, 30001, 6, 80, 40, False, True, True), (B16, 4001, 10, 80, 6, False, False, False),    # vectors of one element
    (H16, 9007, 17, 72, 20, True, False, False), (F32, 7001, 9, 72, 70, True, False, True)])
def test_rope(attn, dtype, T, H, D, rot, inter, inverse, in_place):  # noqa: F811
    assert T * H * vectors(dtype, D, rot, inter, in_place) >= 152 * 1024 * (8 if inter else 4)
    g = torch.Generator(device=DEV).manual_seed(T + rot)
    whole = torch.randn((T, (H + 1) * D), generator=g, device=DEV).to(dtype)
    before = whole.clone()
    x = whole[:, D:].unflatten(1, (H, D))                            # behind another head: a token stride of its own
    pos = torch.randint(0, 700, (T,), generator=g, device=DEV).to(torch.int32)
    tab = attn.rope_table(700, rot, device=DEV)
    ref, big = turned(x, pos, tab, inter, inverse), 2 * x.double().abs().amax(-1, keepdim=True)
    out = attn.rope(x, pos, tab, interleaved=inter, inverse=inverse, out=x if in_place else None)
    assert torch.equal(out[..., rot:], before[:, D:].unflatten(1, (H, D))[..., rot:]), "the unturned part is copied"
    assert not ((out.double() - ref).abs() > U[dtype] * ref.abs() + 4 * 2.0 ** -24 * big).any()
    assert torch.equal(whole[:, :D], before[:, :D]) and (in_place or torch.equal(whole, before))


# layers, K/V heads, query heads (0: none), head_dim, rot (0: no rotation), interleaved, new tokens
APPENDS = [(B16, 1, 3, 7, 80, 24, False, 9000), (H16, 1, 1, 5, 128, 128, False, 12000), (B16, 1, 2, 9, 64, 32, True, 20000),
           (H16, 1, 5, 8, 72, 70, True, 9000), (B16, 9, 3, 0, 96, 48, False, 3000), (H16, 7, 5, 0, 128, 128, True, 3000),
           (B16, 33, 3, 0, 128, 0, False, 1100), (H16, 1, 2, 11, 256, 256, False, 4000)]


@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append(attn, i):  # noqa: F811
    """Against rope() bit for bit, v and the rest of the cache as they were; among the sequences a skipped one, and rows of none."""
    dtype, L, H, qh, D, rot, inter, T = APPENDS[i]
    assert T * L * (2 * H + qh) * (vectors(dtype, D, rot, inter) if rot else D // 8) >= 152 * 1024 * (4 if rot and not inter else 8)
    g = torch.Generator(device=DEV).manual_seed(i)
    ps, width = 16, 2 * H + qh
    lens, cu = [37, 0, 500], [11, T // 3, T // 3 + 5, T - 2]           # rows before cu[0] and from cu[-1] on: of no sequence
    pages = sum(-(-(n + b - a) // ps) for n, a, b in zip(lens, cu, cu[1:])) + 4
    cache = attn.KVCache.create(L, pages, ps, H, D, 4, pages, dtype, DEV)
    cache.pool.copy_(torch.randn(cache.pool.shape, generator=g, device=DEV))
    seqs = i32([2, 0, 1])
    assert cache.extend(seqs, i32(lens)).tolist() == [0, 0, 0]
    start = cache.extend(seqs, i32([b - a for a, b in zip(cu, cu[1:])]))
    assert start.tolist() == lens
    start[1] = -1
    qkv = torch.randn((L, T, width, D), generator=g, device=DEV).to(dtype)
    q, k, v = qkv.split([qh, H, H], 2)
    args = {}
    if rot:
        pos = torch.randint(0, 300, (T,), generator=g, device=DEV).to(torch.int32)
        args = dict(pos=pos, cos_sin=attn.rope_table(300, rot, device=DEV), interleaved=inter)
    want = cache.pool.clone()
    for s, a, b, n in ((2, cu[0], cu[1], lens[0]), (1, cu[2], cu[3], lens[2])):
        at = n + torch.arange(b - a, device=DEV)
        page, slot = cache.table[s].long()[at // ps], at % ps
        for layer in range(L):
            kk = k[layer, a:b]
            if rot:
                kk = attn.rope(kk, args["pos"][a:b].clone(), args["cos_sin"], interleaved=inter)
            want[layer, page, 0, :, slot] = kk
            want[layer, page, 1, :, slot] = v[layer, a:b]
    if qh:
        out = cache.append(k[0], v[0], i32(cu), seqs, start, layer=0, q=q[0], **args)
        assert torch.equal(out, attn.rope(q[0], args["pos"], args["cos_sin"], interleaved=inter))
    else:
        assert cache.append(k, v, i32(cu), seqs, start, layer=None, **args) is None
    assert torch.equal(cache.pool.view(torch.int16), want.view(torch.int16))
