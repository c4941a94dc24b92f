"""Compaction with entries that are out of order, repeated or too large, and of many tokens in caches of either launch form."""
import random

import pytest
import torch

from _helpers import have_gpu
from test_gpu_kv import attn, i32, make, same  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]


def moves(ref, q, start, keep):
    """The definition, on the oracle's cache: entry j moves to offset j if it is above the entry before it and in range."""
    for j, i in enumerate(keep):
        if (j and i <= keep[j - 1]) or not j <= i < ref.lens[q] - start:
            continue
        p, x = ref.at(q, start + i)
        p2, x2 = ref.at(q, start + j)
        ref.pool[:, p2, :, :, x2] = ref.pool[:, p, :, :, x].clone()
    ref._cut(q, start + len(keep))


# few 16-byte pieces of a token's rows in all layers (16): one launch; many (2560): one for the moves
SHAPES = [dict(layers=2, H=2, D=16), dict(layers=20, H=4, D=128)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("keep", [[5, 3], [4, 4], [2, 9, 5, 6, 7], [7, 7, 7, 8], [30, 40, 1], [3, 40, 41], [0, 0, 5], [19], [20], [1, -1, 6],
                                  [2 ** 31 - 1, 3], [6, 2 ** 31 - 1, 9]])
def test_entries_that_move_nothing(attn, shape, keep):  # noqa: F811
    cache, ref = make(attn, ps=8, slots=3, max_pages=9, pages=40, **shape)
    cache.extend(i32([1, 0]), i32([33, 9]))
    ref.extend([1, 0], [33, 9])
    cache.compact(i32([1]), i32([13]), i32([0, len(keep)]), i32(keep))           # 20 tokens from 13 on
    moves(ref, 1, 13, keep)
    same(cache, ref, str(keep))


@pytest.mark.parametrize("shape,ps", [(SHAPES[0], 16), (SHAPES[1], 16), (dict(layers=3, H=8, D=256), 32)])
def test_many_tokens_of_several_sequences(attn, shape, ps):  # noqa: F811
    """More entries than a block's table of moves holds, ragged, every layer compared."""
    r = random.Random(ps)
    lens, start = [420, 7, 300, 129, 640, 1], [3, 0, 40, 0, 100, 0]
    cache, ref = make(attn, ps=ps, slots=7, max_pages=-(-640 // ps), pages=sum(-(-n // ps) for n in lens) + 3, **shape)
    seqs = [4, 0, 6, 2, 1, 5]
    cache.extend(i32(seqs), i32(lens))
    ref.extend(seqs, lens)
    keeps = [sorted(r.sample(range(n - s), k)) for n, s, k in zip(lens, start, [200, 3, 128, 129, 391, 0])]
    cache.compact(i32(seqs), i32(start), i32([sum(map(len, keeps[:i])) for i in range(len(keeps) + 1)]), i32(sum(keeps, [])))
    ref.compact(seqs, start, keeps)
    same(cache, ref)
