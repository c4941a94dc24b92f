"""The bounds-checked build on the attention side: ids and positions out of range are reported, and, as in the plain
build, never followed."""
import ctypes

import pytest
import torch

from _helpers import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
DEV = "cuda:0"


@pytest.fixture(scope="module")
def M():
    from weight_only_int4_route_gb300 import build, moe
    build.build_all()
    return moe


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("checked", [False, True])
def test_pages_and_positions(M, checked):
    from weight_only_int4_route_gb300 import attn
    L = M.lib_checked() if checked else M.lib()
    c = attn.KVCache.create(1, 8, 16, 2, 64, 2, 4, torch.bfloat16, DEV)
    c.pool.normal_()
    seqs, cu, start = i32([0]), i32([0, 3]), c.extend(i32([0]), i32([40]))
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    take = lambda: M.check_status(DEV, L)  # noqa: E731
    assert take() == (0, 0)
    q = torch.randn((3, 4, 64), device=DEV).to(torch.bfloat16)
    out, ws = torch.empty_like(q), torch.empty(128 << 20, dtype=torch.uint8, device=DEV)
    start = i32([37])

    def attention():
        return L.moe_attention(c._d, c._p, 0, q.data_ptr(), 256, 4, 3, cu.data_ptr(), seqs.data_ptr(), start.data_ptr(), 1,
                               None, 0, 0.125, out.data_ptr(), None, ws.data_ptr(), ws.numel(), st)

    assert attention() == 0 and take() == (0, 0)
    for bad in (8, 2 ** 31 - 1, -7):
        c.table[0, 1] = bad
        assert attention() == 0
        status, flags = take()
        assert (status, flags) == ((-5, 8) if checked else (0, 0))
        assert torch.isfinite(out).all(), "an unusable page reads as zeros"
    k = torch.randn((3, 2, 64), device=DEV).to(torch.bfloat16)
    before, at = c.pool.clone(), i32([20])
    r = M.KvRows(k=k.data_ptr(), v=k.data_ptr(), k_token_stride=128, v_token_stride=128, cu=cu.data_ptr(), seqs=seqs.data_ptr(),
                 start=at.data_ptr(), n=1, T=3)
    assert L.moe_kv_append(c._d, c._p, 0, 1, ctypes.byref(r), st) == 0
    assert take() == ((-5, 8) if checked else (0, 0))
    assert torch.equal(c.pool, before)
    tab = attn.rope_table(4, 64, device=DEV)
    pos = i32([0, 4, -1])
    assert L.moe_rope(q.data_ptr(), M.BF16, 3, 4, 64, 256, 64, pos.data_ptr(), tab.data_ptr(), 4, 64, 0, 0, out.data_ptr(), 256,
                      64, st) == 0
    assert take() == ((-5, 16) if checked else (0, 0))
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1:]).all()
