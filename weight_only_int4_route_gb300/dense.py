"""The dense operators around experts and attention (include/moe.h, last part): norm of the residual stream with 8-bit rows,
products of 8-bit integers, log probabilities of logits.

A thin binding in the manner of `attn`: shapes checked, outputs and workspaces allocated on the input's device, the work
enqueued on torch's current stream.  A call's tensors are all on the current GPU; others are refused.

    n = rmsnorm(x, weight, residual=stream, q8=True)        # n.sum is the new stream
    qkv = linear_w8a8(n.q, n.scale, w, w_scale)
    logits = linear_w8a8(n.q, n.scale, head, head_scale, out_dtype=torch.float32)
    s = token_logprobs(logits, drafted, k=8)

Rows are the first dimension; the last one is contiguous, rows may lie any stride apart.  The library takes vectors (weights,
scales, biases) and ids that start on 16 bytes: slices that start elsewhere are copied for it.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import attn
from .attn import _i32
from .moe import _TORCH2MOE, _check, _dt, lib

_f32, _i8 = torch.float32, torch.int8
_raw_stream = torch._C._cuda_getCurrentRawStream


class Normed(NamedTuple):
    y: Optional[torch.Tensor]       # (T, d) of x's type
    q: Optional[torch.Tensor]       # int8 (T, d)
    scale: Optional[torch.Tensor]   # fp32 (T,)
    sum: Optional[torch.Tensor]     # x + residual


class Scores(NamedTuple):
    logprob: torch.Tensor           # fp32, of ids' shape
    entropy: torch.Tensor           # fp32 (T,)
    lse: torch.Tensor               # fp32 (T,)
    top_ids: Optional[torch.Tensor]         # int32 (T, k)
    top_logprob: Optional[torch.Tensor]     # fp32 (T, k)


def _device(t: torch.Tensor) -> int:
    dev = t.get_device()
    assert dev >= 0, "tensors are on the GPU"
    assert dev == attn._current_device(), "tensors are on the current GPU"
    return dev


def _rows(t: torch.Tensor, dev: int):
    """(rows, row length, row stride) of a tensor whose rows are contiguous."""
    assert t.get_device() == dev, "a call's tensors are on one GPU"
    n, d = t.shape
    row, one = t.stride()
    assert one == 1 or d == 1, "a row's elements lie side by side"
    return n, d, row if n > 1 else d       # torch leaves the stride of a dimension of one open


def _start(t: torch.Tensor, held: list) -> int:
    """Where t lies, or a copy of it that starts on 16 bytes, kept in `held` until the call has been made."""
    p = t.data_ptr()
    if p & 15:
        held.append(t.clone())
        p = held[-1].data_ptr()
    return p


def _vector(t: torch.Tensor, dev: int, n: int, dtype, held: list) -> int:
    assert t.get_device() == dev, "a call's tensors are on one GPU"
    assert t.dtype is dtype and t.shape == (n,) and t.is_contiguous()
    return _start(t, held)


def rmsnorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
            y: bool = True, q8: bool = False, sum_out: Optional[torch.Tensor] = None) -> Normed:
    """(x + residual) / rms * weight of rows x (T, d): as y in x's type and / or, with q8, as int8 rows q with a scale each.
    With a residual the sum is returned too, in sum_out if given (which may be residual or x itself)."""
    dev = _device(x)
    T, d, xs = _rows(x, dev)
    rp = sp = yp = qp = cp = total = out = q = scale = None
    held = []
    rs = ss = 0
    where = x.device
    if residual is not None:
        assert residual.shape == x.shape and residual.dtype is x.dtype
        rp, rs = residual.data_ptr(), _rows(residual, dev)[2]
        if sum_out is None:
            total, ss = torch.empty((T, d), dtype=x.dtype, device=where), d
        else:
            total, ss = sum_out, _rows(sum_out, dev)[2]
            assert total.shape == x.shape and total.dtype is x.dtype
        sp = total.data_ptr()
    else:
        assert sum_out is None, "sum_out comes with a residual"
    wp = None if weight is None else _vector(weight, dev, d, x.dtype, held)
    if y:
        out = torch.empty((T, d), dtype=x.dtype, device=where)
        yp = out.data_ptr()
    if q8:
        q, scale = torch.empty((T, d), dtype=_i8, device=where), torch.empty(T, dtype=_f32, device=where)
        qp, cp = q.data_ptr(), scale.data_ptr()
    _check(lib().moe_rmsnorm(x.data_ptr(), xs, rp, rs, wp, _dt(x), T, d, eps, sp, ss, yp, qp, cp, _raw_stream(dev)), "moe_rmsnorm")
    return Normed(out, q, scale, total)


def quantize_rows(x: torch.Tensor):
    """Rows x (T, d) -> (int8 (T, d), fp32 scales (T,)): x is about q * scale, a row's largest magnitude 127."""
    dev = _device(x)
    T, d, xs = _rows(x, dev)
    q, scale = torch.empty((T, d), dtype=_i8, device=x.device), torch.empty(T, dtype=_f32, device=x.device)
    _check(lib().moe_quantize_rows(x.data_ptr(), xs, _dt(x), T, d, q.data_ptr(), scale.data_ptr(), _raw_stream(dev)),
           "moe_quantize_rows")
    return q, scale


def linear_w8a8(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a (M, K) int8 with scales (M,) times w (N, K) int8 with scales (N,), transposed, plus bias fp32 (N,): (M, N).  Sums are
    exact, a row's result is the same in every batch."""
    dev = _device(a)
    M, K, a_row = _rows(a, dev)
    N, k, w_row = _rows(w, dev)
    assert a.dtype is _i8 and w.dtype is _i8 and k == K
    held = []
    sa, sw = _vector(a_scale, dev, M, _f32, held), _vector(w_scale, dev, N, _f32, held)
    b = None if bias is None else _vector(bias, dev, N, _f32, held)
    if out is None:
        out, out_row = torch.empty((M, N), dtype=out_dtype, device=a.device), N
    else:
        m, n, out_row = _rows(out, dev)
        assert (m, n) == (M, N)
    assert out.dtype in _TORCH2MOE
    L = lib()
    wp = w.data_ptr()
    whole = (K | w_row | wp) % 16 == 0                 # w is read where it is
    size = L.moe_linear_w8a8_workspace_size(M, 0 if whole else N, K)
    ws = torch.empty(size, dtype=torch.uint8, device=a.device) if size else None
    _check(L.moe_linear_w8a8(a.data_ptr(), a_row, sa, wp, w_row, sw, b, M, N, K, out.data_ptr(), out_row, _dt(out),
                             None if ws is None else ws.data_ptr(), size, _raw_stream(dev)), "moe_linear_w8a8")
    return out


def token_logprobs(logits: torch.Tensor, ids: Optional[torch.Tensor] = None, k: int = 0, scale: float = 1.0) -> Scores:
    """Log probabilities under softmax(scale * logits) of rows (T, V): of ids, int32 (T,) or (T, n), and of the k most
    probable tokens (equal logits: the lower id first), with entropy and lse."""
    dev = _device(logits)
    T, V, row = _rows(logits, dev)
    n, ip, shape, held = 0, None, (T, 0), []
    if ids is not None:
        assert ids.get_device() == dev and ids.dtype is _i32 and ids.is_contiguous(), \
            "index tensors are contiguous int32 on the GPU of the call's other tensors"
        assert ids.dim() in (1, 2) and ids.shape[0] == T
        shape = ids.shape
        n, ip = (1 if ids.dim() == 1 else shape[1]), _start(ids, held)
    where = logits.device
    logprob, entropy = torch.empty(shape, dtype=_f32, device=where), torch.empty(T, dtype=_f32, device=where)
    lse = torch.empty_like(entropy)
    top_ids = top = tp = lp = None
    if k > 0:
        top_ids, top = torch.empty((T, k), dtype=_i32, device=where), torch.empty((T, k), dtype=_f32, device=where)
        tp, lp = top_ids.data_ptr(), top.data_ptr()
    _check(lib().moe_token_logprobs(logits.data_ptr(), row, _dt(logits), T, V, scale, ip, n, logprob.data_ptr(), entropy.data_ptr(),
                                    lse.data_ptr(), k, tp, lp, _raw_stream(dev)), "moe_token_logprobs")
    return Scores(logprob, entropy, lse, top_ids, top)
