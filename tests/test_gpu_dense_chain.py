"""The dense operators in a row, as a decoder step uses them: norm of the stream with 8-bit rows, products, scores; eager, on a
stream of its own, captured and replayed, and in the decoding example."""
import os
import sys

import pytest
import torch

from _helpers import have_gpu
from oracle import dense_oracle as D

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
DEV = "cuda:0"


@pytest.fixture(scope="module")
def dense():
    from weight_only_int4_route_gb300 import build, dense, moe
    build.build()
    moe.lib()
    yield dense
    assert moe.device_error(DEV) == 0


def weights(d, f, V, seed=0):
    g = torch.Generator().manual_seed(seed)
    up, down, head = (torch.randn(s, generator=g) / s[1] ** 0.5 for s in ((f, d), (d, f), (V, d)))
    return [tuple(D.quantize_rows(w)) for w in (up, down, head)] + [(1 + 0.1 * torch.randn(d, generator=g)).half()]


def step(dense, x, stream, up, down, head, gain, ids):
    """stream += x; a block of two products on its norm; the vocabulary's scores of the result."""
    a = dense.rmsnorm(x, gain, residual=stream, y=False, q8=True)
    h = dense.linear_w8a8(a.q, a.scale, *up, out_dtype=torch.float16)
    y = dense.linear_w8a8(*dense.quantize_rows(h), *down, out_dtype=torch.float16)
    b = dense.rmsnorm(y, gain, residual=a.sum, y=False, q8=True, sum_out=a.sum)
    logits = dense.linear_w8a8(b.q, b.scale, *head, out_dtype=torch.float32)
    return b.sum, logits, dense.token_logprobs(logits, ids, k=6)


@pytest.mark.parametrize("T", [1, 13, 40, 300])
def test_a_step_against_the_oracle(dense, T):
    """Each operator against the oracle on what the one before it gave: exact where it is exact."""
    d, f, V = 256, 640, 1500
    g = torch.Generator().manual_seed(T)
    up, down, head, gain = weights(d, f, V)
    x, stream = torch.randn((T, d), generator=g).half(), (3 * torch.randn((T, d), generator=g)).half()
    to = lambda p: tuple(t.to(DEV) for t in p)  # noqa: E731
    a = dense.rmsnorm(x.to(DEV), gain.to(DEV), residual=stream.to(DEV), y=False, q8=True)
    assert torch.equal(a.sum.cpu(), (x.float() + stream.float()).half())
    steps, scale = D.steps8(D.rmsnorm(x, stream, gain, 1e-6)[1])
    assert ((a.q.double().cpu() - steps).abs() <= 0.5 + 127 * 6 * 2.0 ** -24).all()
    assert ((a.scale.double().cpu() - scale).abs() <= 48 * 2.0 ** -24 * scale).all()
    h = dense.linear_w8a8(a.q, a.scale, *to(up), out_dtype=torch.float16)
    assert torch.equal(h.cpu(), D.linear_w8a8(a.q.cpu(), a.scale.cpu(), *up, None, torch.float16))
    hq = dense.quantize_rows(h)
    ref = D.quantize_rows(h.cpu())
    assert torch.equal(hq[0].cpu(), ref[0]) and torch.equal(hq[1].cpu(), ref[1])
    logits = dense.linear_w8a8(a.q, a.scale, *to(head), out_dtype=torch.float32)
    assert torch.equal(logits.cpu(), D.linear_w8a8(a.q.cpu(), a.scale.cpu(), *head, None, torch.float32))
    s = dense.token_logprobs(logits, k=6)
    assert torch.equal(s.top_ids.cpu(), D.token_logprobs(logits.cpu(), None, 6)[3])


@pytest.mark.parametrize("T", [2, 50])
def test_a_step_on_another_stream_and_replayed(dense, T):
    d, f, V = 512, 1024, 4000
    g = torch.Generator().manual_seed(T)
    w = [tuple(t.to(DEV) for t in p) if isinstance(p, tuple) else p.to(DEV) for p in weights(d, f, V, 1)]
    xs = [torch.randn((T, d), generator=g).half().to(DEV) for _ in range(4)]
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).to(DEV)
    zero = torch.zeros((T, d), dtype=torch.float16, device=DEV)
    ref, stream = [], zero
    for x in xs:
        stream, logits, s = step(dense, x, stream, *w, ids)
        ref.append([stream.clone(), logits, *s])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        stream = zero
        for x, r in zip(xs, ref):
            stream, logits, s = step(dense, x, stream, *w, ids)
            other.synchronize()
            assert all(torch.equal(p, q) for p, q in zip([stream, logits, *s], r))
    torch.cuda.synchronize()
    x_in, s_in = xs[0].clone(), zero.clone()
    graphs, held = [], []
    for _ in range(2):                                       # two graphs of the same tensors
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(step(dense, x_in, s_in, *w, ids))
        graphs.append(graph)
    for x, r in zip(xs, ref):
        x_in.copy_(x)
        for graph, (stream, logits, s) in zip(graphs, held):
            graph.replay()
            assert all(torch.equal(p, q) for p, q in zip([stream, logits, *s], r))
        s_in.copy_(held[0][0])


def test_the_example_with_8_bit_projections(dense):
    """What its rounds leave in the cache is what one causal pass over the same tokens gives."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import speculative_decode as E

    prompts = [[3, 1, 4, 1, 5], [9] * 33, [2, 6]]
    m, cache, out, accepted, _ = E.generate(prompts, rounds=3, int8=True)
    n = len(prompts)
    kept = [sum(a[b] for a in accepted) for b in range(n)]
    assert cache.lens.tolist() == [len(p) + k for p, k in zip(prompts, kept)]
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
        # layer 0: norm and products of a row are the same bits in every batch
        assert torch.equal(a[0], r[0])
        assert torch.isfinite(a).all() and torch.isfinite(r).all()
