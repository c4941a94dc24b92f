"""A workspace of moe_attention_workspace_size serves every call of fewer tokens or sequences (host side only)."""
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
