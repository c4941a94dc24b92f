"""Products of 8-bit integers on the GPU: the oracle's whole-number sums and single fp32 operations, bit for bit."""
import numpy as np
import pytest
import torch

from _helpers import have_gpu
from oracle import dense_oracle as D

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
DEV = "cuda:0"
I8 = torch.int8


@pytest.fixture(scope="module")
def dense():
    from weight_only_int4_route_gb300 import build, dense, moe
    build.build()
    moe.lib()
    yield dense
    assert moe.device_error(DEV) == 0


def draw(M, N, K, seed=0, lo=-128, hi=128):
    g = torch.Generator().manual_seed(seed * 7919 + M * 31 + N * 17 + K)
    i8 = lambda *s: torch.randint(lo, hi, s, generator=g, dtype=torch.int16).to(I8)  # noqa: E731
    f = lambda n: torch.rand(n, generator=g) * 0.02 + 1e-3  # noqa: E731
    return i8(M, K), f(M), i8(N, K), f(N), torch.randn(N, generator=g)


def same(a, b):
    return torch.equal(a.cpu().view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.view(torch.int16 if b.element_size() == 2 else torch.int32))


SIZES = [  # M, N, K
    (1, 1, 1), (1, 16, 16), (1, 17, 33), (1, 6144, 4096), (3, 40, 256), (7, 100, 272), (8, 4096, 512), (9, 64, 1408), (16, 48, 4096),
    (17, 130, 640), (31, 999, 2048), (32, 128, 128), (33, 128, 128), (33, 16, 16), (40, 1000, 1024), (64, 129, 144), (65, 257, 4096),
    (100, 1, 2048), (128, 128, 1040), (129, 384, 2064), (191, 300, 1008), (192, 256, 4112), (193, 520, 384), (200, 77, 48), (300, 640, 5632),
    (385, 128, 100), (512, 1024, 1024), (1000, 333, 767), (1111, 5001, 1408), (2048, 2048, 2048)]


@pytest.mark.parametrize("dtype,with_bias", [(torch.bfloat16, False), (torch.float16, True), (torch.float32, True)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(dense, M, N, K, dtype, with_bias):
    a, sa, w, sw, b = draw(M, N, K)
    b = b if with_bias else None
    got = dense.linear_w8a8(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), None if b is None else b.to(DEV), out_dtype=dtype)
    assert same(got, D.linear_w8a8(a, sa, w, sw, b, dtype))


@pytest.mark.parametrize("M,N,K", [(2, 20, 131071), (40, 130, 131071), (40, 130, 131056), (200, 256, 20000), (24, 40, 65536)])
@pytest.mark.parametrize("fill", ["lowest", "random", "alternating"])
def test_long_sums_are_exact(dense, M, N, K, fill):
    """Sums far past 2^24, where fp32 would round: every value -128 (the largest sum there is), large random ones, and large
    partial sums that cancel."""
    a, sa, w, sw, _ = draw(M, N, K, lo=90)
    if fill == "lowest":
        a, w = torch.full_like(a, -128), torch.full_like(w, -128)
    if fill == "alternating":
        a[:, K // 2:] *= -1
    one = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    got = dense.linear_w8a8(a.to(DEV), one[0], w.to(DEV), one[1], out_dtype=torch.float32)
    acc = (a.double() @ w.double().T)
    assert torch.equal(got.cpu(), torch.from_numpy(acc.to(torch.int32).numpy().astype(np.float32)))


def test_a_rows_result_is_the_same_in_every_batch(dense):
    a, sa, w, sw, b = (t.to(DEV) for t in draw(700, 384, 2304))
    whole = dense.linear_w8a8(a, sa, w, sw, b, out_dtype=torch.float32)
    for rows in (1, 5, 12, 30, 33, 48, 100, 190, 250, 511):
        for first in (0, 700 - rows):
            part = dense.linear_w8a8(a[first:first + rows], sa[first:first + rows].clone(), w, sw, b, out_dtype=torch.float32)
            assert torch.equal(part, whole[first:first + rows]), rows


@pytest.mark.parametrize("M", [1, 5, 20, 60, 300])
@pytest.mark.parametrize("how", ["a", "w", "out", "odd", "bytes"])
def test_strides(dense, M, how):
    """Rows apart, rows that do not start on 16 bytes, results inside a wider tensor."""
    N, K = 150, 192
    a, sa, w, sw, b = draw(M, N, K)
    wide = torch.full((M + 2, 400), 7.0, device=DEV, dtype=torch.bfloat16)
    first = 101 if how == "odd" else 96
    out = wide[1:M + 1, first:first + N] if how in ("out", "odd") else None
    ga, gw = a.to(DEV), w.to(DEV)
    if how in ("a", "odd"):
        big = torch.full((M, K + 64), 99, dtype=I8, device=DEV)
        ga = big[:, 16:16 + K].copy_(ga)
    if how == "w":
        big = torch.full((N, K + 64), 99, dtype=I8, device=DEV)
        gw = big[:, 32:32 + K].copy_(gw)
    if how == "bytes":
        ga = torch.full((M, K + 7), 99, dtype=I8, device=DEV)[:, 3:3 + K].copy_(ga)
        gw = torch.full((N, K + 5), 99, dtype=I8, device=DEV)[:, 1:1 + K].copy_(gw)
    got = dense.linear_w8a8(ga, sa.to(DEV), gw, sw.to(DEV), b.to(DEV), out=out)
    assert same(got.contiguous(), D.linear_w8a8(a, sa, w, sw, b, torch.bfloat16))
    if out is not None:
        assert got is out
        rest = torch.ones_like(wide, dtype=torch.bool)
        rest[1:M + 1, first:first + N] = False
        assert (wide[rest] == 7).all()


@pytest.mark.parametrize("M", [3, 50, 400])
def test_scales_that_are_not_finite(dense, M):
    """A row whose scale is NaN (a row that could not be quantized) gives NaN in all its products and nothing elsewhere."""
    a, sa, w, sw, _ = draw(M, 140, 256)
    a[1], sa[1] = 0, float("nan")
    got = dense.linear_w8a8(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), out_dtype=torch.float32).cpu()
    assert torch.isnan(got[1]).all()
    keep = [i for i in range(M) if i != 1]
    assert same(got[keep], D.linear_w8a8(a[keep], sa[keep], w, sw, None, torch.float32))


@pytest.mark.parametrize("M,N,K", [(4, 64, 512), (60, 256, 1024), (60, 250, 1000), (500, 384, 2048)])
def test_the_workspace_s_contents_have_no_influence(dense, M, N, K):
    import ctypes  # noqa: F401
    from weight_only_int4_route_gb300 import moe
    L = moe.lib()
    a, sa, w, sw, b = (t.to(DEV) for t in draw(M, N, K))
    size = L.moe_linear_w8a8_workspace_size(M + 100, N, K)     # of more rows
    res = []
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((size + 256,), fill, dtype=torch.uint8, device=DEV)
        out = torch.empty((M, N), dtype=torch.float32, device=DEV)
        assert L.moe_linear_w8a8(a.data_ptr(), K, sa.data_ptr(), w.data_ptr(), K, sw.data_ptr(), b.data_ptr(), M, N, K, out.data_ptr(), N, 2,
                                 ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert (ws[size:] == fill).all()
        res.append(out)
    assert torch.equal(res[0], res[1]) and torch.equal(res[0], res[2])


def test_repeats_on_two_streams_agree(dense):
    """Two calls at once, each with a workspace of its own, many times over."""
    a, sa, w, sw, b = (t.to(DEV) for t in draw(260, 512, 3000))
    ref = dense.linear_w8a8(a, sa, w, sw, b)
    few = dense.linear_w8a8(a[:6], sa[:6].clone(), w, sw, b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for i in range(40):
        with torch.cuda.stream(streams[i % 2]):
            outs.append((dense.linear_w8a8(a, sa, w, sw, b), dense.linear_w8a8(a[:6], sa[:6].clone(), w, sw, b)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref) and torch.equal(y, few) for x, y in outs)


@pytest.mark.parametrize("M", [4, 48, 333])
def test_captured_and_replayed(dense, M):
    a, sa, w, sw, b = (t.to(DEV) for t in draw(M, 384, 1536))
    x = torch.zeros_like(a)
    dense.linear_w8a8(x, sa, w, sw, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dense.linear_w8a8(x, sa, w, sw, b)
    for _ in range(3):
        x.copy_(torch.roll(x, 1, 0) if bool(x.any()) else a)
        graph.replay()
        assert torch.equal(out, dense.linear_w8a8(x, sa, w, sw, b))


def test_results_past_32_bits(dense):
    """More results than 2^31: rows at the end are what they are in a small batch."""
    M, N, K = 70001, 32000, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    a = torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int16).to(I8)
    w = torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int16).to(I8)
    sa, sw = torch.rand(M, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    whole = dense.linear_w8a8(a, sa, w, sw)
    for first in (0, 35000, M - 9):
        part = dense.linear_w8a8(a[first:first + 9], sa[first:first + 9].clone(), w, sw)
        assert torch.equal(part, whole[first:first + 9])
    assert same(part, D.linear_w8a8(a[-9:].cpu(), sa[-9:].cpu(), w.cpu(), sw.cpu(), None, torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(190, 19456, 384), (64, 8192, 1536), (1000, 2048, 640)])
def test_many_launches_agree(dense, M, N, K):
    """Hundreds of launches with everything of a CTA's pipeline at its start: rows in memory before weights are converted, other
    weights each time."""
    sets = [tuple(t.to(DEV) for t in draw(M, N, K, seed)[:4]) for seed in range(4)]
    refs = [dense.linear_w8a8(a, sa, w, sw, out_dtype=torch.float32) for a, sa, w, sw in sets]
    few = [dense.linear_w8a8(a[:16], sa[:16].clone(), w, sw, out_dtype=torch.float32) for a, sa, w, sw in sets]    # another kernel
    assert all(torch.equal(r[:16], f) for r, f in zip(refs, few))
    bad = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(400):
        a, sa, w, sw = sets[i % 4]
        bad += (dense.linear_w8a8(a, sa, w, sw, out_dtype=torch.float32) != refs[i % 4]).sum()
    assert int(bad) == 0
