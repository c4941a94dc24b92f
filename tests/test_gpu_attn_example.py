"""The decoding example end to end: what its rounds leave in the cache is what one causal pass over the same tokens
gives."""
import os
import sys

import pytest
import torch

from _helpers import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]


def test_speculative_decode_example():
    from weight_only_int4_route_gb300 import build, moe
    build.build()
    moe.lib()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import speculative_decode as E

    prompts = [[3, 1, 4, 1, 5], [9] * 33, [2, 6]]
    m, cache, out, accepted, counts = E.generate(prompts, rounds=3)
    assert moe.device_error("cuda:0") == 0
    rounds, n = len(accepted), len(prompts)
    kept = [sum(a[b] for a in accepted) for b in range(n)]
    assert cache.lens.tolist() == [len(p) + k for p, k in zip(prompts, kept)]
    assert [len(o) for o in out] == [k + 1 for k in kept]
    assert int(cache.refs.sum()) == sum(-(-x // 16) for x in cache.lens.tolist())
    # a draft row counts once per layer and expert: k experts a row
    assert counts.sum().item() == rounds * n * 10 * m.cfg.k * len(m.blocks)
    # one causal pass over prompt + kept tokens into a fresh cache
    whole = [p + o[:-1] for p, o in zip(prompts, out)]
    lens = [len(w) for w in whole]
    fresh = E.attn.KVCache.create(len(m.blocks), 64, 16, m.kv_heads, m.head_dim, n, 16, m.cfg.torch_dtype, E.DEV)
    seqs = E.ints(list(range(n)))
    start = fresh.extend(seqs, E.ints(lens))
    pos = torch.cat([torch.arange(x, dtype=torch.int32) for x in lens]).to(E.DEV)
    m.forward(torch.tensor(sum(whole, []), device=E.DEV), fresh, E.ints([sum(lens[:i]) for i in range(n + 1)]), seqs, start, pos)
    for b in range(n):
        rows = [c.pool[:, c.table[b, :-(-lens[b] // 16)].long()].transpose(1, 2).float() for c in (cache, fresh)]
        a, r = (x.transpose(2, 3).flatten(3, 4)[:, :, :, :lens[b]] for x in rows)   # layers, 2, heads, tokens, head_dim
        # layer 0's K and V are functions of the tokens alone and of their positions: one f16 rounding apart at most;
        # later layers carry the attention's and the experts' f16 roundings of two different batch shapes
        assert torch.allclose(a[0], r[0], rtol=2.0 ** -9, atol=2.0 ** -9)
        assert float((a - r).norm() / r.norm()) < 2e-2
