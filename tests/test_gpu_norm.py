"""Norm of rows and rows in 8 bits on the GPU against the float64 oracle.

Bounds, in units of e = 2^-24 (half a step of fp32).  h = x + residual is rounded once.  The sum of squares: a thread adds up
to 32 squares, its warp 5 times, the row's warps up to 32 times, so 69 roundings at most, halved by the root; the mean's
product and eps 2, halved; rsqrtf 2 ulp (4 e); h's own rounding in its square, halved twice: 1.  So the factor is off by at most 41 e
and v = h r w, with h's rounding and two products, by 44 e: 48 e below.  y is then rounded to its type (u).  The scale is max|h w| (3
roundings) / 127 (1) times the factor: 45 e, 48 e below.  A code is h w times 127 / max|h w|: h, the product, the maximum's two and the
division's and the last product's roundings, 6 e of at most 127, before it is rounded to the nearest integer."""
import math

import numpy as np
import pytest
import torch

from _helpers import have_gpu
from oracle import dense_oracle as D

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
E = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def dense():
    from weight_only_int4_route_gb300 import build, dense, moe
    build.build()
    moe.lib()
    return dense


def draw(T, d, dtype, seed, pad=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, d + pad), generator=g) * scale).to(dtype)[:, :d]


def on(t):
    """The same strides on the GPU."""
    return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=DEV).copy_(t)


def check(n, x, residual, weight, eps):
    h, v = D.rmsnorm(x, residual, weight, eps)
    if n.sum is not None:
        assert torch.equal(n.sum.cpu(), (x.float() + residual.float()).to(x.dtype)), "the sum: one addition, one rounding"
    if n.y is not None:
        # f16's subnormal steps are 2^-24 wide
        bound = (U[x.dtype] + 48 * E) * v.abs() + (2.0 ** -25 if x.dtype is torch.float16 else 0)
        assert ((n.y.double().cpu() - v).abs() <= bound).all()
    if n.q is not None:
        steps, scale = D.steps8(v)
        assert ((n.scale.double().cpu() - scale).abs() <= 48 * E * scale).all()
        assert ((n.q.double().cpu() - steps).abs() <= 0.5 + 127 * 6 * E).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,d,pad,with_residual,with_weight", [
    (1, 1, 0, True, True), (3, 8, 0, True, True), (5, 7, 1, True, True), (130, 64, 0, False, True), (9, 128, 8, True, False), (2, 129, 0, True, True),
    (33, 1000, 24, True, True), (200, 1408, 0, True, True), (4, 2047, 0, False, False), (301, 2048, 512, True, True), (2, 4096, 4, True, True),
    (7, 5120, 0, True, True), (3, 6145, 0, True, True), (3, 8192, 0, True, True), (2, 8200, 0, True, True), (1, 16384, 0, True, True),
    (2, 16383, 0, True, True), (160, 16384, 0, False, True), (1, 3, 0, False, False)])
def test_norm(dense, dtype, T, d, pad, with_residual, with_weight):
    x = draw(T, d, dtype, T + d, pad)
    residual = draw(T, d, dtype, d, 0, 4.0) if with_residual else None
    weight = (1 + 0.2 * draw(1, d, torch.float32, 7)[0]).to(dtype) if with_weight else None
    args = (on(x), None if weight is None else on(weight), 1e-5)
    r = None if residual is None else on(residual)
    check(dense.rmsnorm(*args, residual=r, y=True, q8=True), x, residual, weight, 1e-5)
    only = dense.rmsnorm(*args, residual=r, y=False, q8=True)
    assert only.y is None and (only.sum is None) == (r is None)
    check(only, x, residual, weight, 1e-5)
    check(dense.rmsnorm(*args, residual=r), x, residual, weight, 1e-5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [96, 4096, 333])
def test_in_place(dense, dtype, d):
    x, residual, weight = draw(6, d, dtype, 1), draw(6, d, dtype, 2, 8), draw(1, d, dtype, 3)[0]
    ref = dense.rmsnorm(on(x), on(weight), residual=on(residual), q8=True)
    for target in ("residual", "x"):
        t = dict(x=on(x), residual=on(residual))
        n = dense.rmsnorm(t["x"], on(weight), residual=t["residual"], q8=True, sum_out=t[target])
        assert n.sum is t[target] and torch.equal(t[target], ref.sum)
        assert torch.equal(n.y, ref.y) and torch.equal(n.q, ref.q) and torch.equal(n.scale, ref.scale)


def test_neighbours_are_left_alone(dense):
    """sum_out inside a wider tensor, and at an odd element: what lies around it stays."""
    x, residual = draw(5, 40, torch.bfloat16, 1), draw(5, 40, torch.bfloat16, 2)
    for first in (8, 3):
        wide = torch.full((7, 64), 3.0, dtype=torch.bfloat16, device=DEV)
        out = wide[1:6, first:first + 40]
        n = dense.rmsnorm(on(x), residual=on(residual), sum_out=out)
        check(n, x, residual, None, 1e-6)
        rest = torch.ones_like(wide, dtype=torch.bool)
        rest[1:6, first:first + 40] = False
        assert (wide[rest] == 3).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_a_row_does_not_depend_on_the_others(dense, dtype):
    """Alone, among a few and among many rows: the same bits, on every run."""
    for d in (96, 1024, 4096, 8200, 333):
        x, r = draw(400, d, dtype, 5), draw(400, d, dtype, 6)
        many = dense.rmsnorm(on(x), residual=on(r), q8=True)
        for first, n in ((0, 1), (7, 20), (399, 1), (100, 300), (0, 400)):
            part = dense.rmsnorm(on(x[first:first + n]), residual=on(r[first:first + n]), q8=True)
            assert all(torch.equal(a[first:first + n], b) for a, b in zip(many, part))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_and_small_values(dense, dtype):
    """Squares past fp32's range, rows near its lower end, rows of zeros."""
    x = draw(6, 512, dtype, 9)
    x = torch.stack([x[0] * 1e19, x[1] * 1e30, x[2] * 1e-18, x[3] * 1e-30, x[4] * 0, x[5]])
    n = dense.rmsnorm(on(x), q8=True)
    h, v = D.rmsnorm(x, None, None, 1e-6)
    fine = torch.tensor([0, 1, 2, 5])                        # the others' results are below fp32's normal numbers or zero
    bound = (U[dtype] + 48 * E) * v.abs()
    assert ((n.y.double().cpu() - v).abs() <= bound)[fine].all()
    steps, scale = D.steps8(v)
    assert ((n.scale.double().cpu() - scale).abs() <= 48 * E * scale)[fine].all()
    assert ((n.q.double().cpu() - steps).abs() <= 0.5 + 127 * 6 * E).all()
    assert n.scale[4] == 0 and (n.q[4] == 0).all() and (n.y[4] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 2048])
def test_no_eps(dense, dtype, d):
    """Without an eps rows of any size are normalised, squares below fp32's numbers included; a row of zeros is 0 / 0."""
    x = draw(5, d, dtype, 19) * torch.tensor([[1.0], [2.0 ** -40], [2.0 ** -64], [2.0 ** -100], [0.0]]).to(dtype)
    n = dense.rmsnorm(on(x), None, 0.0, q8=True)
    v = D.rmsnorm(x, None, None, 0.0)[1]
    steps, scale = D.steps8(torch.nan_to_num(v))
    assert ((n.y.double().cpu() - v).abs() <= (U[dtype] + 48 * E) * v.abs())[:4].all() and torch.isnan(n.y[4]).all()
    assert ((n.scale.double().cpu() - scale).abs() <= 48 * E * scale).all()
    assert ((n.q.double().cpu() - steps).abs() <= 0.5 + 127 * 6 * E).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d", [64, 2048, 77])
def test_rows_that_are_not_finite(dense, dtype, bad, d):
    x = draw(4, d, dtype, 11)
    x[1, d // 3] = bad
    n = dense.rmsnorm(on(x), q8=True)
    q, s = dense.quantize_rows(on(x))
    for codes, scale in ((n.q, n.scale), (q, s)):
        assert (codes[1] == 0).all() and torch.isnan(scale[1])
        assert torch.isfinite(scale[[0, 2, 3]]).all() and (codes[[0, 2, 3]].abs().amax(1) == 127).all()
    y = n.y[1].float().cpu()
    if math.isnan(bad):
        assert torch.isnan(y).all()
    else:                                                    # x / inf = 0, inf / inf = NaN
        assert torch.isnan(y[d // 3]) and int((y == 0).sum()) == d - 1
    keep = torch.tensor([0, 2, 3])
    check(n._replace(y=n.y[keep], q=n.q[keep], scale=n.scale[keep]), x[keep], None, None, 1e-6)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,d,pad", [(1, 1, 0), (4, 31, 0), (65, 256, 8), (3, 5632, 0), (300, 2048, 0), (2, 16384, 0), (5, 9001, 0)])
def test_quantize_rows_is_exact(dense, dtype, T, d, pad):
    """Single fp32 operations, so the same bits as the oracle's."""
    x = draw(T, d, dtype, d, pad, 3.0)
    if d > 8:
        x[0, 1:] = 0
        x[-1] *= 2.0 ** -14                                  # f16: down to its subnormal numbers
    q, s = dense.quantize_rows(on(x))
    rq, rs = D.quantize_rows(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)


def test_tiny_rows_quantize(dense):
    x = draw(3, 64, torch.float32, 3) * torch.tensor([[2.0 ** -120], [2.0 ** -135], [2.0 ** 120]])
    q, s = dense.quantize_rows(on(x))
    rq, rs = D.quantize_rows(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)


def test_many_rows(dense):
    """More rows than a launch dimension's 65535."""
    x = torch.randn((70001, 24), generator=torch.Generator().manual_seed(2)).to(torch.float16)
    q, s = dense.quantize_rows(x.to(DEV))
    assert torch.equal(s.cpu(), torch.from_numpy(x.float().abs().amax(1).numpy() / np.float32(127)))
    assert (q.abs().amax(1) == 127).all()


def test_rows_past_32_bits(dense):
    """Rows whose offsets pass 2^31 elements."""
    T, d = 1100, 16
    wide = torch.empty((T, 2 ** 21), dtype=torch.bfloat16, device=DEV)
    x = draw(T, d, torch.bfloat16, 4)
    wide[:, :d] = x.to(DEV)
    q, s = dense.quantize_rows(wide[:, :d])
    rq, rs = D.quantize_rows(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)


def test_elements_past_32_bits(dense):
    T, d = 140001, 16384
    x = torch.randn((T, d), dtype=torch.bfloat16, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    n = dense.rmsnorm(x, q8=True)
    for first in (0, 70000, T - 3):
        part = dense.rmsnorm(x[first:first + 3], q8=True)
        assert torch.equal(part.y, n.y[first:first + 3]) and torch.equal(part.q, n.q[first:first + 3])
        check(part, x[first:first + 3].cpu(), None, None, 1e-6)
