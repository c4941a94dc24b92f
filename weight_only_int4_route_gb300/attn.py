"""Rotary positions, the paged key/value cache and attention over it (include/moe.h, second half).

The attention half of a decoder layer beside the expert layer of `moe`: a thin binding in the same manner (shapes
checked, outputs and workspaces allocated on the input's device, the work enqueued on torch's current stream).

    cache = KVCache.create(layers, pages, page_size, kv_heads, head_dim, slots, max_pages, dtype)
    start = cache.extend(seqs, n_new)                       # once per step, for every layer
    mask, pos = tree_mask(parents, cu, start, max_draft)
    q = cache.append(k, v, cu, seqs, start, layer, q=q, pos=pos, cos_sin=table)
    out = attention(q, cache, cu, seqs, start, mask=mask, layer=layer)
    cache.compact(seqs, start, cu_keep, keep)               # keep the accepted path
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
from typing import Optional

import torch

from .moe import KvDesc, KvPointers, KvRows, _check, _dt, _ptr, _stream, lib

SCALING = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


def _ints(*tensors):
    for t in tensors:
        assert t.dtype == torch.int32 and t.is_contiguous(), "index tensors are contiguous int32"


def rope_table(n_pos: int, rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original: int = 0, device="cuda:0") -> torch.Tensor:
    """Cosines and sines of positions 0 .. n_pos - 1: fp32 (n_pos, rot), the first half of a row the cosines."""
    out = torch.empty((n_pos, rot), dtype=torch.float32, device=device)
    _check(lib().moe_rope_table(n_pos, rot, base, SCALING[scaling], factor, original, _ptr(out), _stream(out.device)),
           "moe_rope_table")
    return out


def rope(x: torch.Tensor, pos: torch.Tensor, cos_sin: torch.Tensor, interleaved: bool = False, inverse: bool = False,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x (T, heads, head_dim), any token and head strides, turned by its positions; inverse=True turns back, which
    is the gradient.  out=x works in place."""
    T, H, D = x.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    _ints(pos)
    assert x.stride(2) == 1 and out.stride(2) == 1 and out.shape == x.shape and out.dtype == x.dtype
    assert pos.shape == (T,) and cos_sin.dtype == torch.float32 and cos_sin.is_contiguous()
    _check(lib().moe_rope(_ptr(x), _dt(x), T, H, D, x.stride(0), x.stride(1), _ptr(pos), _ptr(cos_sin), cos_sin.shape[0],
                          cos_sin.shape[1], int(interleaved), int(inverse), _ptr(out), out.stride(0), out.stride(1),
                          _stream(x.device)), "moe_rope")
    return out


@dataclasses.dataclass
class KVCache:
    """The cache's tensors: pool (layers, pages, 2, kv_heads, page_size, head_dim), table (slots, max_pages), lens
    (slots,), refs (pages,)."""
    pool: torch.Tensor
    table: torch.Tensor
    lens: torch.Tensor
    refs: torch.Tensor

    def __post_init__(self):
        L, P, two, H, ps, D = self.pool.shape
        S, W = self.table.shape
        _ints(self.table, self.lens, self.refs)
        assert two == 2 and self.pool.is_contiguous() and self.lens.shape == (S,) and self.refs.shape == (P,)
        self.desc = KvDesc(L, P, ps, H, D, S, W, _dt(self.pool))
        self.ptrs = KvPointers(self.pool.data_ptr(), self.table.data_ptr(), self.lens.data_ptr(), self.refs.data_ptr())
        self._d, self._p = ctypes.byref(self.desc), ctypes.byref(self.ptrs)

    @staticmethod
    def create(layers: int, pages: int, page_size: int, kv_heads: int, head_dim: int, slots: int, max_pages: int,
               dtype: torch.dtype = torch.bfloat16, device="cuda:0") -> "KVCache":
        """An empty cache (the pool's contents are left as they are)."""
        i32 = dict(dtype=torch.int32, device=device)
        return KVCache(torch.empty((layers, pages, 2, kv_heads, page_size, head_dim), dtype=dtype, device=device),
                       torch.full((slots, max_pages), -1, **i32), torch.zeros(slots, **i32), torch.zeros(pages, **i32))

    def _st(self):
        return _stream(self.pool.device)

    def extend(self, seqs: torch.Tensor, n_new: torch.Tensor) -> torch.Tensor:
        """Grow sequences `seqs` by `n_new` tokens; returns their lengths before (all -1 if the pages do not suffice:
        nothing has changed then)."""
        _ints(seqs, n_new)
        assert seqs.shape == n_new.shape
        n = seqs.numel()
        start = torch.empty_like(seqs)
        ws = torch.empty(max(16, int(lib().moe_kv_extend_workspace_size(self._d, n))), dtype=torch.uint8, device=seqs.device)
        _check(lib().moe_kv_extend(self._d, self._p, _ptr(seqs), _ptr(n_new), n, _ptr(start), _ptr(ws), ws.numel(),
                                   self._st()), "moe_kv_extend")
        return start

    def fork(self, src: torch.Tensor, dst: torch.Tensor) -> None:
        """Empty slots `dst` become copies of `src` that share their pages until they are written to."""
        _ints(src, dst)
        assert src.shape == dst.shape
        _check(lib().moe_kv_fork(self._d, self._p, _ptr(src), _ptr(dst), src.numel(), self._st()), "moe_kv_fork")

    def free(self, seqs: torch.Tensor) -> None:
        _ints(seqs)
        _check(lib().moe_kv_free(self._d, self._p, _ptr(seqs), seqs.numel(), self._st()), "moe_kv_free")

    def compact(self, seqs: torch.Tensor, start: torch.Tensor, cu_keep: torch.Tensor, keep: torch.Tensor) -> None:
        """Of the tokens from start[i] on keep those at the ascending offsets keep[cu_keep[i]:cu_keep[i+1]]."""
        _ints(seqs, start, cu_keep, keep)
        n = seqs.numel()
        assert start.shape == seqs.shape and cu_keep.numel() == n + 1
        _check(lib().moe_kv_compact(self._d, self._p, _ptr(seqs), _ptr(start), _ptr(cu_keep), _ptr(keep), keep.numel(), n,
                                    self._st()), "moe_kv_compact")

    def copy(self, src: torch.Tensor, dst: torch.Tensor) -> None:
        """Pages `src` -> `dst` on every layer."""
        _ints(src, dst)
        assert src.shape == dst.shape
        _check(lib().moe_kv_copy(self._d, self._p, _ptr(src), _ptr(dst), src.numel(), self._st()), "moe_kv_copy")

    def append(self, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, seqs: torch.Tensor, start: torch.Tensor,
               layer: Optional[int] = 0, q: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
               cos_sin: Optional[torch.Tensor] = None, interleaved: bool = False) -> Optional[torch.Tensor]:
        """Write the new tokens' k and v (T, kv_heads, head_dim) into `layer`, or with layer=None into every layer from
        (layers, T, kv_heads, head_dim).  With cos_sin, k is rotated on its way, and q too if given (returned)."""
        L, T = (1, k.shape[0]) if layer is not None else k.shape[:2]
        H, D = self.desc.kv_heads, self.desc.head_dim
        _ints(cu, seqs, start)
        n = seqs.numel()
        assert start.shape == seqs.shape and cu.numel() == n + 1 and k.shape == v.shape and k.shape[-2:] == (H, D)
        assert k.dim() == (3 if layer is not None else 4) and (layer is not None or L == self.desc.layers)
        assert k.dtype == v.dtype == self.pool.dtype and k.stride()[-2:] == v.stride()[-2:] == (D, 1)
        r = KvRows(k=k.data_ptr(), v=v.data_ptr(), k_token_stride=k.stride(-3), v_token_stride=v.stride(-3),
                   k_layer_stride=0 if layer is not None else k.stride(0), v_layer_stride=0 if layer is not None else v.stride(0),
                   cu=cu.data_ptr(), seqs=seqs.data_ptr(), start=start.data_ptr(), n=n, T=T)
        out = None
        if cos_sin is not None:
            _ints(pos)
            assert pos.shape == (T,) and cos_sin.dtype == torch.float32 and cos_sin.is_contiguous()
            r.cos_sin, r.pos, r.n_pos, r.rot, r.interleaved = cos_sin.data_ptr(), pos.data_ptr(), *cos_sin.shape, int(interleaved)
        if q is not None:
            assert q.dim() == 3 and q.shape[0] == T and q.shape[2] == D and q.stride()[1:] == (D, 1) and q.dtype == k.dtype
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            r.q, r.q_token_stride, r.q_heads, r.q_out = q.data_ptr(), q.stride(0), q.shape[1], out.data_ptr()
        _check(lib().moe_kv_append(self._d, self._p, layer or 0, L, ctypes.byref(r), self._st()), "moe_kv_append")
        return out


def tree_mask(parents: torch.Tensor, cu: torch.Tensor, start: torch.Tensor, max_draft: int):
    """Trees of drafted tokens, given by each token's parent within its sequence (-1: the context) -> (mask, pos):
    each token's visible drafted tokens as bits, int32 (T, ceil(max_draft / 32)), and its position."""
    _ints(parents, cu, start)
    T, words = parents.numel(), max(1, -(-max_draft // 32))
    assert cu.numel() == start.numel() + 1
    mask = torch.empty((T, words), dtype=torch.int32, device=parents.device)
    pos = torch.empty(T, dtype=torch.int32, device=parents.device)
    _check(lib().moe_tree_mask(_ptr(parents), _ptr(cu), _ptr(start), start.numel(), T, words, _ptr(mask), _ptr(pos),
                               _stream(parents.device)), "moe_tree_mask")
    return mask, pos


def attention(q: torch.Tensor, cache: KVCache, cu: torch.Tensor, seqs: torch.Tensor, start: torch.Tensor,
              mask: Optional[torch.Tensor] = None, layer: int = 0, scale: Optional[float] = None,
              return_lse: bool = False):
    """Attention of the new tokens q (T, q_heads, head_dim), already in the cache from start[i] on: causal, or with
    `mask` (tree_mask) over drafted trees.  Returns out, or (out, lse) with lse fp32 (T, q_heads)."""
    T, H, D = q.shape
    _ints(cu, seqs, start)
    n = seqs.numel()
    assert start.shape == seqs.shape and cu.numel() == n + 1
    assert D == cache.desc.head_dim and q.dtype == cache.pool.dtype and q.stride()[1:] == (D, 1)
    words = 0
    if mask is not None:
        _ints(mask)
        assert mask.dim() == 2 and mask.shape[0] == T
        words = mask.shape[1]
    out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if return_lse else None
    wsb = int(lib().moe_attention_workspace_size(cache._d, T, n, H))
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=q.device)
    _check(lib().moe_attention(cache._d, cache._p, layer, _ptr(q), q.stride(0), H, T, _ptr(cu), _ptr(seqs), _ptr(start), n,
                               _ptr(mask), words, 1.0 / math.sqrt(D) if scale is None else scale, _ptr(out), _ptr(lse),
                               _ptr(ws), ws.numel(), _stream(q.device)), "moe_attention")
    return (out, lse) if return_lse else out
