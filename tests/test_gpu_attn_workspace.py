"""moe_attention's workspace: what it holds before a call has no influence, and one sized for a call serves smaller ones."""
import ctypes
import math

import pytest
import torch

from _helpers import have_gpu
from test_gpu_attention import B16, DEV, H16, Case, attn, i32  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]


def call(c, ws):
    from weight_only_int4_route_gb300 import moe
    q, cu, seqs, start = c.q.to(DEV), i32(c.cu), i32(c.slots), i32(c.ctx)
    T, H, D = q.shape
    out = torch.full((T, H, D), math.nan, dtype=q.dtype, device=DEV)
    lse = torch.full((T, H), math.nan, device=DEV)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    status = moe.lib().moe_attention(c.cache._d, c.cache._p, c.layer, q.data_ptr(), H * D, H, T, cu.data_ptr(), seqs.data_ptr(),
                                     start.data_ptr(), len(c.new), None, 0, D ** -0.5, out.data_ptr(), lse.data_ptr(),
                                     ws.data_ptr(), ws.numel(), st)
    torch.cuda.synchronize()
    return status, out, lse


CASES = {
    "one_row_tile_split": (B16, 8, 2, 128, 16, [1, 5, 30], [9000, 100, 2500]),
    "one_row_tile_whole": (H16, 4, 4, 64, 16, [3] * 300, [20] * 300),
    "two_row_tiles": (B16, 8, 2, 128, 64, [1500, 200], [30, 700]),
    "two_row_tiles_short": (H16, 8, 8, 64, 16, [300], [0]),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_contents_have_no_influence(attn, name):  # noqa: F811
    from weight_only_int4_route_gb300 import moe
    c = Case(attn, *CASES[name], seed=41)
    T, H = c.q.shape[:2]
    need = moe.lib().moe_attention_workspace_size(c.cache._d, T, len(c.new), H)
    got = []
    for fill in (0, 0xFF, 0x7F, 0x01):
        status, out, lse = call(c, torch.full((need,), fill, dtype=torch.uint8, device=DEV))
        assert status == 0
        got.append((out, lse))
    c.check(*got[0])
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


def test_a_workspace_serves_smaller_calls(attn):  # noqa: F811
    """Sized for 64 tokens of 64 sequences, it serves 64 tokens of one (the form with two row tiles, which needs more)."""
    from weight_only_int4_route_gb300 import moe
    many, one = (Case(attn, B16, 4, 1, 64, 16, *a, seed=42) for a in (([1] * 64, [9] * 64), ([64], [9])))
    need = moe.lib().moe_attention_workspace_size(many.cache._d, 64, 64, 4)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    for c in (many, one):
        status, out, lse = call(c, ws)
        assert status == 0, moe.lib().moe_last_error_string()
        c.check(out, lse)
