"""The attention oracle against values worked out by hand, and the host-side refusals of the attention-side calls
(no GPU: every call here is refused, or does nothing, before a launch)."""
import ctypes
import math

import pytest
import torch

from oracle import attn_oracle as A
from weight_only_int4_route_gb300 import build as B
from weight_only_int4_route_gb300 import moe as M


def test_rope_quarter_turn():
    """rot = 2: one frequency of 1; a table row of 90 degrees maps (a, b) to (-b, a), the rest is copied."""
    t = torch.tensor([[0.0, 1.0]])
    x = torch.tensor([[[3.0, 5.0, 7.0, 9.0]]])
    assert A.rope(x, torch.tensor([0]), t).tolist() == [[[-5.0, 3.0, 7.0, 9.0]]]
    assert A.rope(x, torch.tensor([0]), t, inverse=True).tolist() == [[[5.0, -3.0, 7.0, 9.0]]]
    t4 = torch.tensor([[0.0, 1.0, 1.0, 0.0]])         # first pair turned, second not
    assert A.rope(x, torch.tensor([0]), t4).tolist() == [[[-7.0, 5.0, 3.0, 9.0]]]
    assert A.rope(x, torch.tensor([0]), t4, interleaved=True).tolist() == [[[-5.0, 3.0, 7.0, 9.0]]]


def test_rope_scalings():
    plain, one = A.rope_frequencies(64)
    assert plain[0] == 1.0 and one == 1.0
    lin, _ = A.rope_frequencies(64, scaling="linear", factor=4.0)
    assert all(abs(a / b - 4.0) < 1e-12 for a, b in zip(plain, lin))
    ntk, _ = A.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and abs(plain[-1] / ntk[-1] - 4.0) < 1e-9
    parts, m = A.rope_frequencies(64, scaling="parts", factor=4.0, original=4096)
    assert parts[0] == 1.0 and abs(plain[-1] / parts[-1] - 4.0) < 1e-12 and abs(m - (0.1 * math.log(4.0) + 1)) < 1e-15


def test_rope_gradient_is_the_inverse():
    """d/dx of <g, rope(x)> equals rope(g, inverse): by central differences."""
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randn((2, 1, 8), generator=g, dtype=torch.float64) for _ in range(2))
    pos, tab = torch.tensor([3, 11]), A.rope_table(range(16), 6)
    grad = A.rope(w, pos, tab, inverse=True)
    for t in range(2):
        for d in range(8):
            e = torch.zeros_like(x)
            e[t, 0, d] = 1e-3
            diff = ((A.rope(x + e, pos, tab) - A.rope(x - e, pos, tab)) * w).sum() / 2e-3
            assert abs(float(diff - grad[t, 0, d])) < 1e-10


def test_cache_oracle_by_hand():
    pool = torch.arange(6 * 4, dtype=torch.float64).reshape(1, 6, 1, 1, 4, 1).repeat(1, 1, 2, 1, 1, 1)
    c = A.Cache(pool, slots=3, max_pages=3)
    assert c.extend([0], [5]) == [0] and c.table[0] == [0, 1] and c.refs == [1, 1, 0, 0, 0, 0]
    c.fork([0], [1])
    assert c.refs == [2, 2, 0, 0, 0, 0]
    assert c.extend([1, 0], [1, 0]) == [5, 5]                      # page 1 is copied to 2, its other holder keeps it
    assert c.table[1] == [0, 2] and c.refs == [2, 1, 1, 0, 0, 0]
    assert torch.equal(c.pool[:, 2], c.pool[:, 1])
    assert c.extend([0], [99]) == [-1] and c.lens == [5, 6, 0]     # past max_pages: nothing changes
    c.compact([1], [4], [[1]])                                     # token 5 moves to 4
    assert c.lens[1] == 5 and float(c.pool[0, 2, 0, 0, 0]) == 5.0
    c.compact([1], [4], [[]])
    assert c.table[1] == [0] and c.refs == [2, 1, 0, 0, 0, 0]
    c.free([0, 1])
    assert c.refs == [0] * 6


def test_tree_mask_by_hand():
    see, pos = A.tree_mask([-1, 0, 0, 2, -2, 4, -1], [0, 7], [10], 1)
    assert see == [{0}, {0, 1}, {0, 2}, {0, 2, 3}, set(), set(), {6}]
    assert pos == [10, 11, 11, 12, 10, 10, 10]
    assert A.bits([{0, 31}, {33}], 2).tolist() == [[1 - (1 << 31), 0], [0, 2]]


def test_attention_by_hand():
    """Two visible keys with scores 0 and ln 3: weights 1/4 and 3/4; a key that is not visible may hold NaN."""
    q = torch.tensor([[[1.0]], [[1.0]]])
    k = torch.tensor([[[0.0], [math.log(3.0)], [math.nan]]])
    v = torch.tensor([[[4.0], [8.0], [math.nan]]])
    out, lse, _, _ = A.attention(q, k, v, [[0, 1], []], 1.0)
    assert abs(float(out[0]) - 7.0) < 1e-6 and abs(float(lse[0]) - math.log(4.0)) < 1e-6
    assert float(out[1]) == 0.0 and float(lse[1]) == -math.inf


# ---------------------------------------------------------------- refusals


@pytest.fixture(scope="module")
def L():
    B.build()
    return M.lib()


P = ctypes.c_void_p(0x1000)
BAD = ctypes.c_void_p(0x1004)
NUL = ctypes.c_void_p(0)


def desc(**kw):
    d = dict(layers=2, pages=64, page_size=16, kv_heads=4, head_dim=64, slots=8, max_pages=8, dtype=M.BF16)
    d.update(kw)
    return M.KvDesc(*(d[f] for f, _ in M.KvDesc._fields_))


def ptrs(**kw):
    d = dict(pool=0x1000, table=0x1000, lens=0x1000, refs=0x1000)
    d.update(kw)
    return M.KvPointers(*(d[f] for f, _ in M.KvPointers._fields_))


@pytest.mark.parametrize("kw", [dict(dtype=M.F32), dict(layers=0), dict(pages=0), dict(pages=1 << 30), dict(page_size=4),
                                dict(page_size=24), dict(page_size=512), dict(kv_heads=0), dict(head_dim=20),
                                dict(head_dim=264), dict(slots=0), dict(max_pages=0), dict(slots=1 << 20, max_pages=1 << 12),
                                dict(max_pages=1 << 20)])
def test_bad_cache_geometry_is_refused(L, kw):
    d, p = desc(**kw), ptrs()
    assert L.moe_kv_extend_workspace_size(ctypes.byref(d), 4) == 0
    assert L.moe_kv_free(ctypes.byref(d), ctypes.byref(p), P, 1, NUL) == -1
    assert L.moe_attention_workspace_size(ctypes.byref(d), 4, 1, 4) == 0


def test_cache_calls_refuse_bad_arguments(L):
    d, p = ctypes.byref(desc()), ctypes.byref(ptrs())
    for bad in (dict(pool=0), dict(table=0x1008), dict(lens=0), dict(refs=0x1004)):
        assert L.moe_kv_fork(d, ctypes.byref(ptrs(**bad)), P, P, 1, NUL) == -1
    assert L.moe_kv_extend(d, p, P, P, 4, P, P, 16, NUL) == -3 and b"workspace" in L.moe_last_error_string()
    assert L.moe_kv_extend(d, p, P, P, 4, P, NUL, 1 << 20, NUL) == -1
    assert L.moe_kv_extend(d, p, P, BAD, 4, P, P, 1 << 20, NUL) == -1
    assert L.moe_kv_extend(d, p, P, P, -1, P, P, 1 << 20, NUL) == -1
    assert L.moe_kv_extend(d, p, NUL, NUL, 0, NUL, NUL, 0, NUL) == 0          # nothing to do
    assert L.moe_kv_copy(d, p, P, NUL, 1, NUL) == -1
    assert L.moe_kv_compact(d, p, P, P, P, NUL, 3, 1, NUL) == -1
    assert L.moe_kv_compact(d, p, P, P, P, P, -1, 1, NUL) == -1
    assert L.moe_kv_free(d, p, NUL, 0, NUL) == 0
    assert L.moe_kv_extend(None, p, P, P, 1, P, P, 1 << 20, NUL) == -1


def rows(**kw):
    d = dict(k=0x1000, v=0x1000, k_token_stride=256, v_token_stride=256, cu=0x1000, seqs=0x1000, start=0x1000, n=1, T=4)
    d.update(kw)
    return ctypes.byref(M.KvRows(**d))


def test_append_refuses_bad_arguments(L):
    d, p = ctypes.byref(desc()), ctypes.byref(ptrs())
    go = lambda layer=0, n=1, **kw: L.moe_kv_append(d, p, layer, n, rows(**kw), NUL)  # noqa: E731
    assert go(layer=2) == -1 and go(layer=1, n=2) == -1 and go(layer=-1) == -1 and go(n=0) == -1
    assert go(k_token_stride=4) == -1 and go(v_token_stride=-8) == -1
    assert go(k=0) == -1 and go(v=0x1008) == -1 and go(cu=0) == -1
    assert go(q=0x1000, q_out=0x2000, q_heads=4, q_token_stride=256) == -1                    # q without cos_sin
    rot = dict(cos_sin=0x1000, pos=0x1000, n_pos=8, rot=64)
    assert go(**{**rot, "rot": 66}) == -1 and go(**{**rot, "rot": 3}) == -1 and go(**{**rot, "pos": 0}) == -1
    assert go(**{**rot, "n_pos": 0}) == -1
    assert go(**rot, q=0x1000, q_out=0x1000, q_heads=4, q_token_stride=256) == -1             # in place
    assert go(n=2, **rot, q=0x1000, q_out=0x2000, q_heads=4, q_token_stride=256) == -1        # two layers
    assert go(T=0) == 0


def test_rope_refuses_bad_arguments(L):
    def go(x=P, dtype=M.BF16, T=4, heads=2, dim=64, xt=128, xh=64, pos=P, tab=P, n_pos=8, rot=64, out=BAD, ot=128, oh=64):
        return L.moe_rope(x, dtype, T, heads, dim, xt, xh, pos, tab, n_pos, rot, 0, 0, out, ot, oh, NUL)
    o = ctypes.c_void_p(0x4000)
    assert go() == -1                                                                          # out misaligned
    assert go(out=o, dtype=5) == -1 and go(out=o, dim=60) == -1 and go(out=o, rot=63) == -1 and go(out=o, rot=66) == -1
    assert go(out=o, xt=132) == -1 and go(out=o, xh=-64) == -1 and go(out=o, n_pos=0) == -1 and go(out=o, pos=NUL) == -1
    assert go(out=o, oh=32) == -1                                                              # heads of out overlap
    assert go(out=P, ot=256) == -1                                                             # in place, other strides
    assert go(out=o, T=0) == 0
    assert L.moe_rope_table(8, 64, 10000.0, 9, 1.0, 0, P, NUL) == -1
    assert L.moe_rope_table(8, 2, 10000.0, 2, 4.0, 0, P, NUL) == -1                            # NTK needs rot > 2
    assert L.moe_rope_table(8, 64, 10000.0, 3, 4.0, 0, P, NUL) == -1                           # PARTS needs original
    assert L.moe_rope_table(8, 64, 10000.0, 1, 0.5, 0, P, NUL) == -1
    assert L.moe_rope_table(8, 64, 1.0, 0, 1.0, 0, P, NUL) == -1
    assert L.moe_rope_table(0, 64, 10000.0, 0, 1.0, 0, NUL, NUL) == 0


def test_attention_refuses_bad_arguments(L):
    p = ctypes.byref(ptrs())

    def go(d=None, layer=0, q=P, qt=512, heads=8, T=4, cu=P, n=1, mask=NUL, words=0, scale=0.125, out=P, lse=NUL, ws=P,
           wsb=1 << 30):
        return L.moe_attention(ctypes.byref(d or desc()), p, layer, q, qt, heads, T, cu, P, P, n, mask, words, scale, out,
                               lse, ws, wsb, NUL)
    assert go(layer=2) == -1 and go(heads=6) == -1 and go(heads=0) == -1 and go(qt=12) == -1
    assert go(d=desc(head_dim=136)) == -2 and go(d=desc(kv_heads=1), heads=129) == -2
    assert go(mask=P, words=0) == -1 and go(mask=P, words=1025) == -1 and go(mask=BAD, words=1) == -1
    assert go(scale=0.0) == -1 and go(scale=math.inf) == -1 and go(scale=math.nan) == -1
    assert go(q=NUL) == -1 and go(out=BAD) == -1 and go(lse=BAD) == -1 and go(cu=NUL) == -1
    assert go(T=0) == 0 and go(n=0) == 0
    assert L.moe_tree_mask(P, P, P, 1, 4, 0, P, P, NUL) == -1 and L.moe_tree_mask(P, P, NUL, 1, 4, 1, P, P, NUL) == -1
    assert L.moe_tree_mask(NUL, P, P, 1, 4, 1, P, P, NUL) == -1 and L.moe_tree_mask(NUL, NUL, NUL, 0, 4, 1, NUL, NUL, NUL) == 0


def test_binding_refuses_wrong_tensors():
    """Host tensors, wrong types and shapes are refused before the library is asked."""
    from weight_only_int4_route_gb300 import attn
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    x, tab = torch.zeros((2, 1, 16)), torch.zeros((4, 16))
    with pytest.raises(AssertionError):
        attn.rope(x, i32(0, 1), tab)
    with pytest.raises(AssertionError):
        attn.KVCache(torch.zeros((1, 4, 2, 1, 8, 16), dtype=torch.bfloat16), i32(-1, -1).reshape(2, 1), i32(0, 0), i32(0, 0, 0, 0))
    with pytest.raises(AssertionError):
        attn.tree_mask(i32(-1), i32(0, 1), i32(0), 1)
