"""moe_attention on the host side: a workspace of moe_attention_workspace_size serves every call of fewer tokens or
sequences; the range of the scale."""
import ctypes

import pytest

from weight_only_int4_route_gb300 import build as B
from weight_only_int4_route_gb300 import moe as M


@pytest.fixture(scope="module")
def L():
    B.build()
    return M.lib()


@pytest.mark.parametrize("head_dim,kv_heads,group", [(128, 8, 4), (64, 16, 1), (72, 1, 128), (8, 2, 5)])
def test_fewer_tokens_or_sequences_need_no_more(L, head_dim, kv_heads, group):
    d = ctypes.byref(M.KvDesc(1, 64, 16, kv_heads, head_dim, 8, 8, M.BF16))
    size = lambda T, n: L.moe_attention_workspace_size(d, T, n, kv_heads * group)  # noqa: E731
    tokens = sorted({1, 2, 31, 32, 33, 64, 127, 128, 129, 1000, 9000})
    for T in tokens:
        for n in (1, 2, 3, 64, 1000):
            assert size(T, n) > 0
            for T2 in (t for t in tokens if t <= T):
                for n2 in (1, 2, 3, 64, 1000):
                    assert size(T2, n2) <= size(T, n), (T, n, T2, n2)
    assert size(0, 1) == 0 and size(1, 0) == 0


def test_scales_that_leave_the_range_are_refused(L):
    """Scores are taken to base 2: scale * log2(e) has to be finite too.  Nothing to do (T = 0), but the arguments are checked."""
    d, p, P = M.KvDesc(1, 64, 16, 4, 64, 8, 8, M.BF16), M.KvPointers(*[0x1000] * 4), ctypes.c_void_p(0x1000)

    def go(scale):
        return L.moe_attention(ctypes.byref(d), ctypes.byref(p), 0, P, 512, 8, 0, P, P, P, 1, None, 0, scale, P, None, P, 1 << 30, None)
    assert go(2.3e38) == 0 and go(1e-30) == 0
    assert go(2.4e38) == -1 and go(3e38) == -1 and go(-1.0) == -1
