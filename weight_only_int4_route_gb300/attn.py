"""Rotary positions, the paged key/value cache and attention over it (include/moe.h, second half).

The attention half of a decoder layer beside the expert layer of `moe`: a thin binding in the same manner (shapes
checked, outputs and workspaces allocated on the input's device, the work enqueued on torch's current stream).  A call's
tensors are all on the current GPU; others are refused.

    cache = KVCache.create(layers, pages, page_size, kv_heads, head_dim, slots, max_pages, dtype)
    start = cache.extend(seqs, n_new)                       # once per step, for every layer
    mask, pos = tree_mask(parents, cu, start, max_draft)
    q = cache.append(k, v, cu, seqs, start, layer, q=q, pos=pos, cos_sin=table)
    out = attention(q, cache, cu, seqs, start, mask=mask, layer=layer)
    cache.compact(seqs, start, cu_keep, keep)               # keep the accepted path

A kernel that gives up on one of its bounded waits leaves its outputs incomplete and says so through moe.device_error.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .moe import KvDesc, KvPointers, KvRows, _check, _dt, lib

SCALING = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}

# These calls are short (a decode step makes a few per layer), so their host side is kept lean: addresses go to ctypes
# as plain integers, and the current stream is read without building a Stream object (2.2 us of a 10 us call).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_i32 = torch.int32


def _device(t: torch.Tensor) -> int:
    """Index of the GPU that holds t.  The library launches on the current one, whatever the stream: with another one
    current its kernels would be given addresses that are not theirs."""
    dev = t.get_device()
    assert dev >= 0, "tensors are on the GPU"
    assert dev == _current_device(), "tensors are on the current GPU"
    return dev


def _on(dev: int, *tensors) -> None:
    for t in tensors:
        assert t.get_device() == dev, "a call's tensors are on one GPU"


def _ints(dev: int, *tensors) -> None:
    for t in tensors:
        assert t.get_device() == dev and t.dtype is _i32 and t.is_contiguous(), \
            "index tensors are contiguous int32 on the GPU of the call's other tensors"


def _scratch(nbytes: int, like: torch.Tensor) -> torch.Tensor:
    return torch.empty(nbytes if nbytes > 16 else 16, dtype=torch.uint8, device=like.device)


def rope_table(n_pos: int, rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original: int = 0, device="cuda:0") -> torch.Tensor:
    """Cosines and sines of positions 0 .. n_pos - 1: fp32 (n_pos, rot), the first half of a row the cosines."""
    out = torch.empty((n_pos, rot), dtype=torch.float32, device=device)
    stream = _raw_stream(_device(out))
    _check(lib().moe_rope_table(n_pos, rot, base, SCALING[scaling], factor, original, out.data_ptr(), stream),
           "moe_rope_table")
    return out


def rope(x: torch.Tensor, pos: torch.Tensor, cos_sin: torch.Tensor, interleaved: bool = False, inverse: bool = False,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x (T, heads, head_dim), any token and head strides, turned by its positions; inverse=True turns back, which
    is the gradient.  out=x works in place."""
    T, H, D = x.shape
    dev = _device(x)
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    else:
        _on(dev, out)
    _on(dev, cos_sin)
    _ints(dev, pos)
    xt, xh, x1 = x.stride()
    ot, oh, o1 = out.stride()
    if T == 1:
        xt = ot = H * D                                # torch leaves the stride of a dimension of one open
    if H == 1:
        xh = oh = D
    assert x1 == 1 and o1 == 1 and out.shape == x.shape and out.dtype == x.dtype
    assert pos.numel() == T and cos_sin.dtype == torch.float32 and cos_sin.is_contiguous()
    n_pos, rot = cos_sin.shape
    _check(lib().moe_rope(x.data_ptr(), _dt(x), T, H, D, xt, xh, pos.data_ptr(), cos_sin.data_ptr(), n_pos, rot,
                          int(interleaved), int(inverse), out.data_ptr(), ot, oh, _raw_stream(dev)), "moe_rope")
    return out


class KVCache:
    """The cache's tensors: pool (layers, pages, 2, kv_heads, page_size, head_dim), table (slots, max_pages), lens
    (slots,), refs (pages,).  Calls that change the cache are ordered by the caller's stream."""

    def __init__(self, pool: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor):
        L, P, two, H, ps, D = pool.shape
        S, W = table.shape
        dev = pool.get_device()
        assert dev >= 0, "tensors are on the GPU"
        _ints(dev, table, lens, refs)
        assert two == 2 and pool.is_contiguous() and lens.numel() == S and refs.numel() == P
        self.pool, self.table, self.lens, self.refs = pool, table, lens, refs
        self.layers, self.kv_heads, self.head_dim = L, H, D
        self.desc = KvDesc(L, P, ps, H, D, S, W, _dt(pool))
        self.ptrs = KvPointers(pool.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr())
        self._d, self._p = ctypes.byref(self.desc), ctypes.byref(self.ptrs)

    @staticmethod
    def create(layers: int, pages: int, page_size: int, kv_heads: int, head_dim: int, slots: int, max_pages: int,
               dtype: torch.dtype = torch.bfloat16, device="cuda:0") -> "KVCache":
        """An empty cache (the pool's contents are left as they are)."""
        i32 = dict(dtype=_i32, device=device)
        return KVCache(torch.empty((layers, pages, 2, kv_heads, page_size, head_dim), dtype=dtype, device=device),
                       torch.full((slots, max_pages), -1, **i32), torch.zeros(slots, **i32), torch.zeros(pages, **i32))

    def extend(self, seqs: torch.Tensor, n_new: torch.Tensor) -> torch.Tensor:
        """Grow sequences `seqs` by `n_new` tokens; returns their lengths before (all -1 if the pages do not suffice:
        nothing has changed then)."""
        dev = _device(self.pool)
        _ints(dev, seqs, n_new)
        n = seqs.numel()
        assert n_new.numel() == n
        L = lib()
        start = torch.empty_like(seqs)
        ws = _scratch(L.moe_kv_extend_workspace_size(self._d, n), seqs)
        _check(L.moe_kv_extend(self._d, self._p, seqs.data_ptr(), n_new.data_ptr(), n, start.data_ptr(), ws.data_ptr(),
                               ws.numel(), _raw_stream(dev)), "moe_kv_extend")
        return start

    def fork(self, src: torch.Tensor, dst: torch.Tensor) -> None:
        """Empty slots `dst` become copies of `src` that share their pages until they are written to."""
        dev = _device(self.pool)
        _ints(dev, src, dst)
        assert src.numel() == dst.numel()
        _check(lib().moe_kv_fork(self._d, self._p, src.data_ptr(), dst.data_ptr(), src.numel(), _raw_stream(dev)),
               "moe_kv_fork")

    def free(self, seqs: torch.Tensor) -> None:
        """Release the sequences' pages; their slots are empty afterwards."""
        dev = _device(self.pool)
        _ints(dev, seqs)
        _check(lib().moe_kv_free(self._d, self._p, seqs.data_ptr(), seqs.numel(), _raw_stream(dev)), "moe_kv_free")

    def compact(self, seqs: torch.Tensor, start: torch.Tensor, cu_keep: torch.Tensor, keep: torch.Tensor) -> None:
        """Of the tokens from start[i] on keep those at the ascending offsets keep[cu_keep[i]:cu_keep[i+1]]."""
        dev = _device(self.pool)
        _ints(dev, seqs, start, cu_keep, keep)
        n = seqs.numel()
        assert start.numel() == n and cu_keep.numel() == n + 1
        _check(lib().moe_kv_compact(self._d, self._p, seqs.data_ptr(), start.data_ptr(), cu_keep.data_ptr(), keep.data_ptr(),
                                    keep.numel(), n, _raw_stream(dev)), "moe_kv_compact")

    def copy(self, src: torch.Tensor, dst: torch.Tensor) -> None:
        """Pages `src` -> `dst` on every layer."""
        dev = _device(self.pool)
        _ints(dev, src, dst)
        assert src.numel() == dst.numel()
        _check(lib().moe_kv_copy(self._d, self._p, src.data_ptr(), dst.data_ptr(), src.numel(), _raw_stream(dev)),
               "moe_kv_copy")

    def append(self, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, seqs: torch.Tensor, start: torch.Tensor,
               layer: Optional[int] = 0, q: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
               cos_sin: Optional[torch.Tensor] = None, interleaved: bool = False) -> Optional[torch.Tensor]:
        """Write the new tokens' k and v (T, kv_heads, head_dim) into `layer`, or with layer=None into every layer from
        (layers, T, kv_heads, head_dim).  With cos_sin, k is rotated on its way, and q too if given (returned)."""
        H, D = self.kv_heads, self.head_dim
        dev = _device(self.pool)
        _ints(dev, cu, seqs, start)
        n = seqs.numel()
        ks, vs, shape = k.stride(), v.stride(), k.shape
        if layer is None:
            assert len(shape) == 4 and shape[0] == self.layers
            layer, L, kl, vl = 0, self.layers, ks[0], vs[0]
            if L == 1:
                kl = vl = 0                                # torch leaves the stride of a dimension of one open
        else:
            assert len(shape) == 3
            L, kl, vl = 1, 0, 0
        T = shape[-3]
        kt, vt = (ks[-3], vs[-3]) if T != 1 else (H * D, H * D)
        _on(dev, k, v)
        assert start.numel() == n and cu.numel() == n + 1 and v.shape == shape and shape[-2:] == (H, D)
        assert k.dtype == v.dtype == self.pool.dtype and ks[-1] == vs[-1] == 1 and (H == 1 or ks[-2] == vs[-2] == D)
        out, rope_args, q_args = None, (None, None, 0, 0, 0), (None, 0, 0, None)
        if cos_sin is not None:
            _ints(dev, pos)
            _on(dev, cos_sin)
            assert pos.numel() == T and cos_sin.dtype == torch.float32 and cos_sin.is_contiguous()
            rope_args = (cos_sin.data_ptr(), pos.data_ptr(), *cos_sin.shape, int(interleaved))
        if q is not None:
            _on(dev, q)
            qs, qh = q.stride(), q.shape[1]
            assert q.shape == (T, qh, D) and qs[2] == 1 and (qh == 1 or qs[1] == D) and q.dtype == k.dtype
            out = torch.empty((T, qh, D), dtype=q.dtype, device=q.device)
            q_args = (q.data_ptr(), qs[0] if T != 1 else qh * D, qh, out.data_ptr())
        r = KvRows(k.data_ptr(), v.data_ptr(), kt, kl, vt, vl, cu.data_ptr(), seqs.data_ptr(), start.data_ptr(), n, T,
                   *rope_args, *q_args)
        _check(lib().moe_kv_append(self._d, self._p, layer, L, ctypes.byref(r), _raw_stream(dev)), "moe_kv_append")
        return out


def tree_mask(parents: torch.Tensor, cu: torch.Tensor, start: torch.Tensor, max_draft: int):
    """Trees of drafted tokens, given by each token's parent within its sequence (-1: the context) -> (mask, pos):
    each token's visible drafted tokens as bits, int32 (T, ceil(max_draft / 32)), and its position.  Rows of no sequence are
    not written."""
    dev = _device(parents)
    _ints(dev, parents, cu, start)
    T, words = parents.numel(), max(1, -(-max_draft // 32))
    assert cu.numel() == start.numel() + 1
    mask = torch.empty((T, words), dtype=_i32, device=parents.device)
    pos = torch.empty(T, dtype=_i32, device=parents.device)
    _check(lib().moe_tree_mask(parents.data_ptr(), cu.data_ptr(), start.data_ptr(), start.numel(), T, words, mask.data_ptr(),
                               pos.data_ptr(), _raw_stream(dev)), "moe_tree_mask")
    return mask, pos


def attention(q: torch.Tensor, cache: KVCache, cu: torch.Tensor, seqs: torch.Tensor, start: torch.Tensor,
              mask: Optional[torch.Tensor] = None, layer: int = 0, scale: Optional[float] = None,
              return_lse: bool = False):
    """Attention of the new tokens q (T, q_heads, head_dim), already in the cache from start[i] on: causal, or with
    `mask` (tree_mask) over drafted trees.  Returns out, or (out, lse) with lse fp32 (T, q_heads); rows of no sequence
    (before cu[0], from cu[-1] on) are not written."""
    T, H, D = q.shape
    qt, qh, q1 = q.stride()
    dev = _device(cache.pool)
    _ints(dev, cu, seqs, start)
    n = seqs.numel()
    _on(dev, q)
    assert start.numel() == n and cu.numel() == n + 1
    assert D == cache.head_dim and q.dtype == cache.pool.dtype and (qh == D or H == 1) and q1 == 1
    words, bits = 0, None
    if mask is not None:
        _ints(dev, mask)
        assert mask.dim() == 2 and mask.shape[0] == T
        words, bits = mask.shape[1], mask.data_ptr()
    if T == 1:
        qt = H * D                                     # torch leaves the stride of a dimension of one open
    L = lib()
    out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if return_lse else None
    ws = _scratch(L.moe_attention_workspace_size(cache._d, T, n, H), q)
    _check(L.moe_attention(cache._d, cache._p, layer, q.data_ptr(), qt, H, T, cu.data_ptr(), seqs.data_ptr(),
                           start.data_ptr(), n, bits, words, D ** -0.5 if scale is None else scale, out.data_ptr(),
                           None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev)),
           "moe_attention")
    return (out, lse) if return_lse else out
