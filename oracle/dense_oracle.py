"""Oracle of the dense operators: norm of rows, rows in 8 bits, products of 8-bit integers, token log probabilities.

Plain CPU code written from the definitions in include/moe.h: float64 where a result is computed in floating point, whole
numbers where it is exact, and fp32 where the definition names single fp32 operations."""
from __future__ import annotations

import math

import numpy as np
import torch


def rmsnorm(x, residual, weight, eps):
    """float64 (h, v)."""
    h = x.double() if residual is None else x.double() + residual.double()
    v = h / ((h * h).mean(1, keepdim=True) + eps).sqrt()
    return h, v if weight is None else v * weight.double()


def steps8(v):
    """float64 rows -> (v * 127 / max|v|, max|v| / 127): codes before rounding, scales.  Rows of zeros give zeros."""
    top = v.abs().amax(1)
    return torch.where(top[:, None] > 0, v * 127 / torch.where(top > 0, top, 1)[:, None], 0), top / 127


def quantize_rows(x):
    """The fp32 operations of the definition, one by one: (int8, fp32)."""
    v = x.float().numpy()
    q, scale = np.zeros(v.shape, np.int8), np.zeros(v.shape[0], np.float32)
    for r in range(v.shape[0]):
        top = np.max(np.abs(v[r]))
        if not np.isfinite(v[r]).all():
            scale[r] = np.nan
        elif top > 0:
            scale[r] = top / np.float32(127)
            up = np.float32(2.0 ** 60 if top < 2.0 ** -60 else 1)
            q[r] = np.rint(v[r] * up * (np.float32(127) / (top * up)))
    return torch.from_numpy(q), torch.from_numpy(scale)


def linear_w8a8(a, a_scale, w, w_scale, bias, dtype):
    """Whole-number sums, then the definition's fp32 operations and one rounding."""
    acc = (a.double() @ w.double().T)                  # exact: sums below 2^53
    assert float(acc.abs().max() if acc.numel() else 0) < 2.0 ** 31
    v = acc.to(torch.int32).numpy().astype(np.float32) * a_scale.numpy()[:, None] * w_scale.numpy()[None, :]
    if bias is not None:
        v = v + bias.numpy()[None, :]
    return torch.from_numpy(v).to(dtype)


def token_logprobs(x, ids, k, scale=1.0):
    """(logprob, entropy, lse, top ids, top logprob), one row at a time."""
    T, V = x.shape
    n = 0 if ids is None else ids.shape[1]
    logprob, entropy, lse = torch.zeros(T, n, dtype=torch.float64), torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    top_ids, top = torch.full((T, k), -1, dtype=torch.int32), torch.full((T, k), -math.inf, dtype=torch.float64)
    for t in range(T):
        row = x[t].double()
        z = row * scale
        m = float(z.max())
        if math.isnan(m) or bool(torch.isnan(z).any()):
            logprob[t], entropy[t], lse[t], top[t] = math.nan, math.nan, math.nan, math.nan
            continue
        if math.isinf(m):
            lse[t], entropy[t] = m, (math.nan if m > 0 else 0.0)
            lp = torch.full_like(z, -math.inf)
            if m > 0:
                lp[z == m] = math.nan
        else:
            total = math.log(float((z - m).exp().sum()))
            lse[t] = m + total
            lp = (z - m) - total                       # rows of a type's lowest value: m + ln V has lost ln V
            entropy[t] = -sum(math.exp(v) * v for v in lp.tolist() if v > -800)
        for i in range(n):
            j = int(ids[t, i])
            logprob[t, i] = lp[j] if 0 <= j < V else math.nan
        order = sorted(range(V), key=lambda j: (-float(row[j]), j))[:k] if V <= 5000 else \
            torch.sort(row, descending=True, stable=True).indices[:k].tolist()
        for i, j in enumerate(order):
            top_ids[t, i], top[t, i] = j, lp[j]
    return logprob, entropy, lse, top_ids, top
