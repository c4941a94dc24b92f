"""A row's norm is the same bits wherever the row lies: alone or in a matrix, at any start and with any stride."""
import pytest
import torch

from _helpers import have_gpu
from test_gpu_norm import DEV, TYPES, dense, draw, on  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]


def same(a, b, rows=slice(None)):
    """The same values; a row of zeros without an eps is 0 / 0 on both sides."""
    return all(p is q or torch.allclose(p[rows].float(), q.float(), rtol=0, atol=0, equal_nan=True) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [8, 96, 256, 264, 1024, 1408, 2048, 4096, 4104, 8200, 16384])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_every_start_and_stride(dense, dtype, d, eps):  # noqa: F811
    T = 9
    x, r, w = draw(T, d, dtype, d), draw(T, d, dtype, d + 1, 0, 4.0), on(draw(1, d, dtype, 3)[0])
    x[2] = (x[2].float() * 2.0 ** -60).to(dtype)                           # without an eps: summed a second time
    r[2] = (r[2].float() * 2.0 ** -60).to(dtype)
    ref = dense.rmsnorm(on(x), w, eps, residual=on(r), q8=True)
    for pad, first in ((1, 0), (8, 0), (8, 3), (5, 2), (16, 1)):
        odd = lambda t: torch.zeros((T, d + pad + 8), dtype=dtype, device=DEV)[:, first:first + d].copy_(t)  # noqa: E731
        for got in (dense.rmsnorm(odd(x), w, eps, residual=on(r), q8=True), dense.rmsnorm(on(x), w, eps, residual=odd(r), q8=True),
                    dense.rmsnorm(on(x), w, eps, residual=on(r), q8=True, sum_out=odd(x * 0))):
            assert same(ref, got), (pad, first)
        rows = odd(x)
        for i in (0, 2, T - 1):
            assert same(ref, dense.rmsnorm(rows[i:i + 1], w, eps, residual=odd(r)[i:i + 1], q8=True), slice(i, i + 1)), (pad, first, i)


def test_the_stride_of_a_single_row_is_not_looked_at(dense):  # noqa: F811
    """Through the C entry point: any number may stand there."""
    from weight_only_int4_route_gb300 import moe
    d = 1024
    x, r = draw(40, d, torch.float32, 1).to(DEV), draw(40, d, torch.float32, 2).to(DEV)
    ref = dense.rmsnorm(x, residual=r, q8=True)
    for i in range(40):
        for stride in (d, 0, -5, 3, d + 1):
            y, q, s, total = torch.empty_like(x[:1]), torch.empty((1, d), dtype=torch.int8, device=DEV), torch.empty(1, device=DEV), torch.empty_like(x[:1])
            assert moe.lib().moe_rmsnorm(x[i].data_ptr(), stride, r[i].data_ptr(), stride, None, 2, 1, d, 1e-6, total.data_ptr(), stride,
                                         y.data_ptr(), q.data_ptr(), s.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
            assert same(ref, (y, q, s, total), slice(i, i + 1))
