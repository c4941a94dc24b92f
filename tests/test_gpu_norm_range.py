"""Norm of rows of any finite size, against the float64 oracle: squares past fp32's largest number for rows up to the type's
largest values.  The bounds are those of test_gpu_norm (the powers of two that a row is taken times are exact); results below the normal numbers are off
by half a subnormal step for each product in fp32 (three of 2^-150) and by half a step of the output's type (bf16: steps of 2^-133,
so 2^-134; fp32 2^-150)."""
import pytest
import torch

from _helpers import have_gpu
from oracle import dense_oracle as D
from test_gpu_norm import E, U, dense, draw, on  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
WIDE = [torch.bfloat16, torch.float32]
LENGTHS = [64, 77, 4096, 16384]


def check(n, x, weight, eps):
    v = D.rmsnorm(x, None, weight, eps)[1]
    half_step = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps / 2
    assert ((n.y.double().cpu() - v).abs() <= (U[x.dtype] + 48 * E) * v.abs() + half_step + 3 * 2.0 ** -150).all()
    steps, scale = D.steps8(v)
    assert ((n.scale.double().cpu() - scale).abs() <= 48 * E * scale).all()
    assert ((n.q.double().cpu() - steps).abs() <= 0.5 + 127 * 6 * E).all()


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("d", LENGTHS)
@pytest.mark.parametrize("with_weight", [False, True])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_rows_up_to_the_largest_values(dense, dtype, d, with_weight, eps):  # noqa: F811
    top = torch.finfo(dtype).max
    row = draw(1, d, torch.float32, 3)[0].clamp(-4, 4) / 4
    x = torch.stack([row * 4e36, row * 4e37, row * top, torch.full((d,), top), torch.full((d,), -top), row]).to(dtype)
    x[5, d // 2] = top
    weight = (1 + 0.2 * draw(1, d, torch.float32, 7)[0].clamp(-3, 3)).to(dtype) if with_weight else None
    check(dense.rmsnorm(on(x), None if weight is None else on(weight), eps, q8=True), x, weight, eps)
