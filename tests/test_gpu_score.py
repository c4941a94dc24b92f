"""Token log probabilities on the GPU against the float64 oracle.

Bounds, in units of e = 2^-24.  A term of Z is 2^t, t = x c - M rounded once: c is off by 2 e relative (the constant's and the
product's roundings), which moves t by 2 e |x c| and, M being a multiple of c too, the term's ratio to the largest by 2 e |t|; t's
rounding e |t|; 2^ itself 4 e.  With |t| 2^t < 0.54 the first two add at most 2 e per term of weight 1, so Z is off by (6 + n) e, n the
roundings on the way to the row's sum: V / 256 (a thread's additions) and 8 + 3 + 3 joins of 4 roundings each.  A log
probability then carries x c's and M's roundings: 4 e of |z_t| and of |z_max|.  S has the same errors term by term, of |t| 2^t, whose sum is
ln 2 (Z's share of the entropy); so the entropy is off by (2 n + 16) e (1 + H) and 4 e of what c's rounding moves in it (|H| and
the spread of z, at most 128 here)."""
import math

import pytest
import torch

from _helpers import have_gpu
from oracle import dense_oracle as D

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
DEV = "cuda:0"
E = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def dense():
    from weight_only_int4_route_gb300 import build, dense, moe
    build.build()
    moe.lib()
    return dense


def check(dense, x, ids, k, scale=1.0):
    where = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEV).copy_(x)
    s = dense.token_logprobs(where, None if ids is None else ids.to(DEV), k=k, scale=scale)
    lp, h, lse, top, toplp = D.token_logprobs(x, None if ids is None else ids.reshape(x.shape[0], -1), k, scale)
    n = x.shape[1] / 256 + 56
    z = x.double() * scale
    big = torch.where(torch.isfinite(z), z.abs(), 0).amax(1)

    def near(got, ref, extra):
        got = got.double().cpu().reshape(ref.shape)
        ref = torch.where(ref.abs() > torch.finfo(torch.float32).max * (1 + E), ref.sign() * math.inf, ref)   # past fp32
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        fine = torch.isfinite(ref)
        assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)])
        bound = (E * (6 + n + extra)).expand(ref.shape) if ref.dim() == 1 else (E * (6 + n + extra))[:, None].expand(ref.shape)
        assert ((got - ref).abs()[fine] <= bound[fine]).all(), float(((got - ref).abs() / bound)[fine].max())

    if ids is not None:
        assert s.logprob.shape == ids.shape
        near(s.logprob, lp, 8 * big)
    near(s.lse, lse, 8 * big)
    near(s.entropy, h, (n + 16) * (1 + torch.nan_to_num(h)) + 4 * 128)
    if k:
        assert torch.equal(s.top_ids.cpu(), top)
        near(s.top_logprob, toplp, 8 * big)
    return s


def draw(T, V, dtype, seed=0, pad=0, spread=2.5):
    g = torch.Generator().manual_seed(seed + T * 13 + V)
    x = (torch.randn((T, V + pad), generator=g) * spread).to(dtype)[:, :V]
    return x, torch.randint(0, V, (T, 3), generator=g, dtype=torch.int32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V,k,pad", [
    (1, 1, 1, 0), (1, 2, 5, 0), (3, 7, 7, 1), (2, 9, 64, 0), (5, 255, 8, 0), (4, 1000, 20, 5), (9, 1003, 33, 0), (2, 4096, 64, 0),
    (1, 32000, 8, 0), (3, 32001, 16, 2), (7, 50001, 17, 0), (1, 131072, 40, 0), (130, 5000, 5, 3), (700, 2049, 8, 0), (650, 9000, 20, 1),
    (6, 65521, 0, 15), (2, 131071, 32, 0)])
def test_scores(dense, dtype, T, V, k, pad):
    x, ids = draw(T, V, dtype, 0, pad)
    check(dense, x, ids, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [2, 800])
@pytest.mark.parametrize("kind", ["equal", "zeros", "steps", "rising", "falling", "masked", "one_group", "peaked", "lowest", "some_lowest",
                                  "few_lanes"])
def test_ties_and_orders(dense, dtype, T, kind):
    """Rows where many logits are equal, sorted rows, rows mostly masked, rows where nearly every logit is above the best one of
    a few threads (the k best are then found one after the other)."""
    V, k = 9600, 12
    j = torch.arange(V).float()
    g = torch.Generator().manual_seed(3)
    row = {"equal": torch.full((V,), 1.5), "zeros": torch.where(j % 2 == 0, -0.0, 0.0), "steps": (j * 7919 % 5),
           "rising": j / 1000, "falling": -j / 1000, "masked": torch.where(j % 4001 == 3, j / 5000, -math.inf),
           "peaked": torch.where(j == 77, 90.0, -20.0), "one_group": torch.randn(V, generator=g),
           "lowest": torch.full((V,), torch.finfo(dtype).min), "few_lanes": torch.randn(V, generator=g),
           "some_lowest": torch.where(j % 1999 == 5, j / 5000, torch.finfo(dtype).min)}[kind]
    if kind == "few_lanes":                                  # all large values are a few threads'
        row = row + torch.where((j // (16 // torch.empty((), dtype=dtype).element_size())) % 256 < 14, 40.0, 0.0)
    if kind == "one_group":
        per = 16 // torch.empty((), dtype=dtype).element_size()
        row = row + torch.where((j // per) % 32 == 31, -30.0, 30.0)
        row = torch.where((j // per) % 256 >= 224, row - 30, row)
    x = row.to(dtype)[None].repeat(T, 1)
    x[1] = torch.roll(x[1], 5)
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    few = [0, 1, T - 1]
    full = dense.token_logprobs(x.to(DEV), ids.to(DEV), k=k)
    check(dense, x[few], ids[few], k)
    lp, h, lse, top, toplp = D.token_logprobs(x[few], ids[few][:, None], k)
    assert torch.equal(full.top_ids[few].cpu(), top)
    assert torch.equal(full.top_ids[2:], full.top_ids[:1].expand(T - 2, k))
    assert torch.allclose(full.top_logprob[few].double().cpu(), toplp, rtol=1e-6, atol=2e-4) and \
        torch.allclose(full.lse[few].double().cpu(), lse, rtol=1e-6, atol=2e-4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(1, 40), (3, 5000), (2, 40000), (800, 700)])
def test_rows_that_are_not_finite(dense, dtype, T, V):
    """Nothing but -inf, one NaN, one and two +inf, all but one masked; beside ordinary rows."""
    for bad in ("empty", "nan", "inf", "infs", "single"):
        x, ids = draw(T, V, dtype, 5)
        if bad == "empty":
            x[0] = -math.inf
        elif bad == "single":
            x[0] = -math.inf
            x[0, V // 3] = 2.5
        else:
            x[0, V // 2] = math.nan if bad == "nan" else math.inf
            if bad == "infs":
                x[0, V - 1] = math.inf
        ids[0, 0] = V // 2
        few = [0, T - 1]
        check(dense, x[few], ids[few], 6)
        if T > 2:
            check(dense, x[:4], ids[:4], 6)
            s = dense.token_logprobs(x.to(DEV), ids.to(DEV), k=6)
            assert torch.isfinite(s.lse[1:]).all() and torch.isfinite(s.logprob[1:]).all()


def test_ids_outside_the_vocabulary(dense):
    x, _ = draw(3, 300, torch.bfloat16)
    s = check(dense, x, torch.tensor([[-1, 0], [299, 300], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32), 0)
    assert torch.isnan(s.logprob).tolist() == [[True, False], [False, True], [True, True]]


@pytest.mark.parametrize("scale", [0.01, 0.7, 3.0])
def test_scale(dense, scale):
    x, ids = draw(5, 3001, torch.float32)
    check(dense, x, ids, 9, scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [1e-30, 1e-5, 1.0, 30.0, 300.0])
def test_masks_beside_the_lowest_values(dense, dtype, scale):
    """-inf has no weight, however near the others are to the type's lowest value and however small the scale is."""
    low = torch.finfo(dtype).min
    x, ids = draw(6, 3000, dtype, 2, spread=1.0 if scale <= 1 else 0.01)
    x[:, 1::3] = -math.inf
    x[1, 0::3] = low
    x[1, 2::3] = -math.inf                                   # a third at the lowest value, nothing else
    x[2] = torch.where(torch.isfinite(x[2]), torch.full((), low, dtype=dtype), x[2])
    x[2, 5] = low / 2
    if dtype is not torch.float16 and scale <= 1:
        x[3, 7], x[4, 8] = 3e38, 2.0 ** 101
    check(dense, x, ids, 7, scale)


def test_forms_of_ids(dense):
    x, ids = draw(4, 500, torch.float16)
    check(dense, x, ids[:, 0].contiguous(), 2)
    assert check(dense, x, None, 2).logprob.shape == (4, 0)
    many = torch.randint(0, 500, (4, 700), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    check(dense, x, many, 0)


@pytest.mark.parametrize("first", [0, 1, 3])
def test_rows_that_start_anywhere(dense, first):
    """Every row at another offset from a 16-byte boundary; what surrounds them is not looked at."""
    for dtype in TYPES:
        x, ids = draw(9, 2005, dtype)
        wide = torch.full((9, 2005 + 12), math.nan, dtype=dtype, device=DEV)[:, :2017]
        flat = torch.full((9 * 2011 + 16,), math.nan, dtype=dtype, device=DEV)
        view = flat[first:first + 9 * 2011].view(9, 2011)[:, :2005]
        view.copy_(x)
        a = dense.token_logprobs(view, ids.to(DEV), k=5)
        b = dense.token_logprobs(wide[:, :2005].copy_(x), ids.to(DEV), k=5)
        assert torch.equal(a.top_ids, b.top_ids) and torch.allclose(a.logprob, b.logprob, rtol=1e-5, atol=1e-5)
        lp = D.token_logprobs(x, ids, 5)
        assert torch.equal(a.top_ids.cpu(), lp[3]) and torch.allclose(a.logprob.double().cpu(), lp[0], rtol=0, atol=1e-4)


def test_rows_past_32_bits(dense):
    T, V = 40, 1500
    wide = torch.empty((T, 2 ** 26), dtype=torch.bfloat16, device=DEV)
    x, ids = draw(T, V, torch.bfloat16)
    wide[:, :V] = x.to(DEV)
    s = dense.token_logprobs(wide[:, :V], ids.to(DEV), k=4)
    lp = D.token_logprobs(x, ids, 4)
    assert torch.equal(s.top_ids.cpu(), lp[3]) and torch.allclose(s.logprob.double().cpu(), lp[0], rtol=0, atol=1e-4)


def test_runs_agree_bit_for_bit_and_replay(dense):
    for T, V in ((2, 60000), (300, 20000), (900, 3000)):
        x, ids = draw(T, V, torch.bfloat16, 8)
        x, ids = x.to(DEV), ids.to(DEV)
        first = dense.token_logprobs(x, ids, k=20)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = dense.token_logprobs(x, ids, k=20)
        for _ in range(20):
            graph.replay()
            again = dense.token_logprobs(x, ids, k=20)
            assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, again, held))


def test_many_short_rows(dense):
    x, ids = draw(200001, 33, torch.bfloat16, 4)
    s = dense.token_logprobs(x.to(DEV), ids.to(DEV), k=3)
    few = torch.tensor([0, 1, 65535, 65536, 131071, 200000])
    lp = D.token_logprobs(x[few], ids[few], 3)
    assert torch.equal(s.top_ids[few].cpu(), lp[3])
    check(dense, x[few], ids[few], 3)
    assert torch.equal(s.logprob[few], dense.token_logprobs(x[few].to(DEV), ids[few].to(DEV), k=3).logprob)
