"""The oracle of the dense operators against values worked out by hand, without a GPU."""
import math

import torch

from oracle import dense_oracle as D


def test_norm_by_hand():
    h, v = D.rmsnorm(torch.tensor([[1.0, 2.0]]), torch.tensor([[2.0, 2.0]]), torch.tensor([1.0, 0.5]), 0.0)
    r = math.sqrt(12.5)                                   # h = (3, 4), mean square 12.5
    assert h.tolist() == [[3.0, 4.0]]
    assert torch.allclose(v, torch.tensor([[3 / r, 2 / r]], dtype=torch.float64), rtol=1e-15)
    steps, scale = D.steps8(v)
    assert torch.allclose(steps, torch.tensor([[127.0, 127 * 2 / 3]], dtype=torch.float64), rtol=1e-15)
    assert math.isclose(float(scale), 3 / r / 127, rel_tol=1e-15)


def test_rows_in_8_bits_by_hand():
    q, s = D.quantize_rows(torch.tensor([[127.0, -0.5, 0.5, 1.5, 2.5], [0.0, 0.0, -0.0, 0.0, 0.0], [1.0, math.inf, 0, 0, 0],
                                         [math.nan, 1.0, 0, 0, 0], [2.0 ** -140, -2.0 ** -140, 0, 2.0 ** -142, 0]]))
    assert q.tolist() == [[127, 0, 0, 2, 2], [0] * 5, [0] * 5, [0] * 5, [127, -127, 0, 32, 0]]    # ties to even, 31.75
    assert s[:2].tolist() == [1.0, 0.0] and torch.isnan(s[2:4]).all()


def test_product_by_hand():
    a, w = torch.tensor([[1, -2, 127]], dtype=torch.int8), torch.tensor([[3, 4, -128], [0, 0, 1]], dtype=torch.int8)
    out = D.linear_w8a8(a, torch.tensor([0.5]), w, torch.tensor([2.0, 0.25]), torch.tensor([1.0, -1.0]), torch.float32)
    assert out.tolist() == [[-(5 + 127 * 128) + 1.0, 127 * 0.125 - 1.0]]


def test_scores_by_hand():
    x = torch.tensor([[0.0, math.log(3.0), -math.inf, 0.0], [-math.inf] * 4, [math.inf, 0, 0, 0], [math.nan, 0, 0, 0]])
    lp, h, lse, top, toplp = D.token_logprobs(x, torch.tensor([[1, 2, 4]] * 4), 3)
    assert torch.allclose(lp[0, 0], torch.tensor(math.log(0.6)).double(), atol=1e-7) and lp[0, 1] == -math.inf and math.isnan(lp[0, 2])
    assert math.isclose(float(h[0]), -(0.6 * math.log(0.6) + 0.4 * math.log(0.2)), rel_tol=1e-6)
    assert math.isclose(float(lse[0]), math.log(5), rel_tol=1e-6)
    assert top[0].tolist() == [1, 0, 3] and top[1].tolist() == [0, 1, 2]            # equal logits: the lower id
    assert lse[1] == -math.inf and h[1] == 0 and (toplp[1] == -math.inf).all() and lp[1, 0] == -math.inf
    assert lse[2] == math.inf and math.isnan(float(h[2])) and lp[2, 0] == -math.inf and math.isnan(float(toplp[2, 0]))
    assert torch.isnan(lse[3]) and top[3].tolist() == [-1] * 3 and torch.isnan(toplp[3]).all()
    half = D.token_logprobs(x[:1] * 2, None, 0, scale=0.5)
    assert math.isclose(float(half[2]), float(lse[0]), rel_tol=1e-12) and half[0].shape == (1, 0)


def test_an_oracle_with_a_planted_mistake_fails_its_pin(monkeypatch):
    monkeypatch.setattr(D.np, "rint", lambda v: D.np.floor(v + 0.5))                # ties upwards
    q, _ = D.quantize_rows(torch.tensor([[127.0, -0.5, 0.5, 1.5, 2.5]]))
    assert q.tolist() != [[127, 0, 0, 2, 2]]
