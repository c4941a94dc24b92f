"""Norm of rows of any finite size, against the float64 oracle: squares past fp32's largest number for rows up to the type's
largest values, and below its smallest for rows down to the smallest subnormal numbers, where there is no eps to cover them.  The
bounds are those of test_gpu_norm (the powers of two that a row is taken times are exact); results below the normal numbers are off
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


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("d", LENGTHS)
def test_rows_down_to_the_smallest_values(dense, dtype, d):  # noqa: F811
    row = draw(1, d, torch.float32, 5)[0]
    x = torch.stack([row * 2.0 ** -100, row * 2.0 ** -116, row * 2.0 ** -126, row * 2.0 ** -126 * 2.0 ** -5, row * 0]).to(dtype)
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    x[4, d // 3] = tiny                                                    # the smallest number there is, alone
    if dtype is torch.float32:
        x = torch.cat([x, torch.stack([row * 2.0 ** -70 * 2.0 ** -66, row * 2.0 ** -70 * 2.0 ** -72, row * 2.0 ** -70 * 2.0 ** -77])])
    check(dense.rmsnorm(on(x), None, 0.0, q8=True), x, None, 0.0)
    assert (x.abs().amax(1) > 0).all()


@pytest.mark.parametrize("dtype", WIDE)
def test_a_small_eps_beside_small_rows(dense, dtype):  # noqa: F811
    """eps between the squares' sizes: it counts whatever power of two a row is taken times."""
    row = draw(1, 512, torch.float32, 6)[0]
    x = torch.stack([row * 2.0 ** -18, row * 2.0 ** -50, row * 2.0 ** -60, row * 2.0 ** -75]).to(dtype)
    for eps in (2.0 ** -40, 2.0 ** -100, 2.0 ** -120, 2.0 ** -149):
        n = dense.rmsnorm(on(x), None, eps, q8=True)
        check(n, x, None, eps)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("d", LENGTHS)
@pytest.mark.parametrize("eps", [1e-6, 1.5, 1e-27])
@pytest.mark.parametrize("with_weight", [False, True])
def test_small_rows_beside_an_eps(dense, dtype, d, eps, with_weight):  # noqa: F811
    """eps covers the squares of rows whose products with the weight are subnormal: the codes and scales are v's all the same.  A
    scale below the normal numbers is rounded once more, by half a step of 2^-149."""
    row = draw(1, d, torch.float32, 8)[0]
    sizes = (2.0 ** -58, 2.0 ** -62, 2.0 ** -100, 2.0 ** -124, 2.0 ** -131) + ((2.0 ** -140, 2.0 ** -147) if dtype is torch.float32 else ())
    x = torch.stack([(row.double() * s).float() for s in sizes] + [row * 0]).to(dtype)
    weight = (1 + 0.2 * draw(1, d, torch.float32, 7)[0].clamp(-3, 3)).to(dtype) if with_weight else None
    n = dense.rmsnorm(on(x), None if weight is None else on(weight), eps, q8=True)
    v = D.rmsnorm(x, None, weight, torch.tensor(eps, dtype=torch.float32).double())[1]
    half_step = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    assert ((n.y.double().cpu() - v).abs() <= (U[dtype] + 48 * E) * v.abs() + half_step + 3 * 2.0 ** -150).all()
    steps, scale = D.steps8(v)
    assert ((n.scale.double().cpu() - scale).abs() <= 48 * E * scale + 2.0 ** -150).all()
    assert ((n.q.double().cpu() - steps).abs() <= 0.5 + 127 * 6 * E).all()
