"""The paged cache on the GPU against the oracle's lists: tables, lengths, holders and contents, all exact."""
import random

import pytest
import torch

from _helpers import have_gpu
from oracle import attn_oracle as A

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
DEV = "cuda:0"


@pytest.fixture(scope="module")
def attn():
    from weight_only_int4_route_gb300 import attn, build, moe
    build.build()
    moe.lib()
    return attn


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(attn, layers=2, pages=40, ps=8, H=2, D=16, slots=7, max_pages=9, dtype=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed)
    pool = torch.randn((layers, pages, 2, H, ps, D), generator=g).to(dtype)
    cache = attn.KVCache.create(layers, pages, ps, H, D, slots, max_pages, dtype, DEV)
    cache.pool.copy_(pool)
    return cache, A.Cache(pool, slots, max_pages)


def same(cache, ref, what=""):
    torch.cuda.synchronize()
    assert cache.lens.tolist() == ref.lens, what
    assert cache.refs.tolist() == ref.refs, what
    assert torch.equal(cache.table.cpu(), ref.table_tensor()), what
    assert torch.equal(cache.pool.cpu().view(torch.int16), ref.pool.view(torch.int16)), what


@pytest.mark.parametrize("ps,D,H,dtype", [(8, 8, 1, torch.float16), (8, 64, 3, torch.bfloat16), (16, 128, 2, torch.bfloat16),
                                          (32, 80, 2, torch.float16), (64, 256, 1, torch.bfloat16), (256, 16, 1, torch.float16)])
def test_a_random_life(attn, ps, D, H, dtype):
    """Random extends, forks, appends, compactions, copies and frees, compared after every call."""
    r = random.Random(ps * D)
    slots, max_pages, pages, layers = 6, 5, 18, 2
    cache, ref = make(attn, layers, pages, ps, H, D, slots, max_pages, dtype, seed=ps)
    g = torch.Generator().manual_seed(9)
    refused = 0
    for step in range(70):
        what = r.choice(["extend", "extend", "fork", "draft", "draft", "free", "copy"])
        seqs = r.sample(range(slots), r.randint(1, slots))
        if what == "extend":
            new = [r.choice([0, 1, ps - 1, ps, ps + 1, r.randint(0, 2 * ps)]) for _ in seqs]
            got, want = cache.extend(i32(seqs), i32(new)).tolist(), ref.extend(seqs, new)
            assert got == want
            refused += want[0] == -1
        elif what == "fork":
            pairs = [(r.randrange(slots), d) for d in seqs]
            dsts = {d for _, d in pairs if ref.lens[d] == 0}
            pairs = [(s, d) for s, d in pairs if s not in dsts]
            cache.fork(i32([s for s, _ in pairs]), i32([d for _, d in pairs]))
            ref.fork([s for s, _ in pairs], [d for _, d in pairs])
        elif what == "draft":
            new = [r.randint(0, ps + 3) for _ in seqs]
            got, start = cache.extend(i32(seqs), i32(new)).tolist(), ref.extend(seqs, new)
            assert got == start
            cu = [sum(new[:i]) for i in range(len(new) + 1)]
            k, v = (torch.randn((layers, cu[-1], H, D), generator=g).to(dtype) for _ in range(2))
            cache.append(k.to(DEV), v.to(DEV), i32(cu), i32(seqs), i32(start), layer=None)
            ref.append(k, v, cu, seqs, start)
            same(cache, ref, f"step {step}: append")
            keeps = [sorted(r.sample(range(m), r.randint(0, m))) for m in new]
            if r.random() < 0.2:
                keeps = [[] for _ in new]
            cache.compact(i32(seqs), i32(start), i32([sum(map(len, keeps[:i])) for i in range(len(new) + 1)]),
                          i32([i for x in keeps for i in x]))
            ref.compact(seqs, start, keeps)
        elif what == "free":
            cache.free(i32(seqs[:2]))
            ref.free(seqs[:2])
        else:
            ids = r.sample(range(pages), 4)
            cache.copy(i32(ids[:2]), i32(ids[2:]))
            for s, d in zip(ids[:2], ids[2:]):
                ref.pool[:, d] = ref.pool[:, s]
        same(cache, ref, f"step {step}: {what}")
    assert 0 < refused, "the life meets a full cache"


def test_shared_page_written_by_all_holders_at_once(attn):
    cache, ref = make(attn)
    for c, f in ((cache, i32), (ref, list)):
        c.extend(f([0]), f([11]))
        c.fork(f([0, 0]), f([1, 2]))
    assert cache.extend(i32([2, 0, 1]), i32([1, 1, 0])).tolist() == ref.extend([2, 0, 1], [1, 1, 0]) == [11, 11, 11]
    same(cache, ref)
    assert cache.extend(i32([1]), i32([1])).tolist() == ref.extend([1], [1])
    same(cache, ref)


def test_many_sequences_and_pages(attn):
    """More sequences and more pages than one block has threads, growth in every length, then all freed."""
    n, pages, ps = 2500, 9000, 8
    cache, ref = make(attn, layers=1, pages=pages, ps=ps, H=1, D=8, slots=n, max_pages=6)
    r = random.Random(2)
    seqs = list(range(n))
    for _ in range(2):
        r.shuffle(seqs)
        new = [r.randint(0, 13) for _ in seqs]
        assert cache.extend(i32(seqs), i32(new)).tolist() == ref.extend(seqs, new)
        same(cache, ref)
    cache.free(i32(seqs[::2]))
    ref.free(seqs[::2])
    some = seqs[:700]
    assert cache.extend(i32(some), i32([20] * 700)).tolist() == ref.extend(some, [20] * 700)
    same(cache, ref)


def test_bad_ids_touch_nothing(attn):
    cache, ref = make(attn)
    assert cache.extend(i32([0, -1, 7, 2 ** 31 - 1, 1]), i32([9, 1, 1, 1, -3])).tolist() == [0, -1, -1, -1, -1]
    ref.extend([0], [9])
    cache.fork(i32([0, -5, 0, 3]), i32([99, 1, 0, -1]))
    cache.free(i32([-1, 7, 2 ** 31 - 1]))
    cache.copy(i32([-1, 40, 3, 4]), i32([1, 2, -7, 4000]))
    k = torch.ones((4, 2, 16), dtype=torch.bfloat16, device=DEV)
    cache.append(k, k, i32([0, 2, 4]), i32([-1, 9]), i32([0, 0]))            # no such slots
    cache.append(k, k, i32([0, 4]), i32([0]), i32([-1]))                     # skipped sequence
    cache.append(k, k, i32([0, 4]), i32([0]), i32([9 * 8 - 2]))              # past the sequence's pages and the table
    cache.append(k, k, i32([4, 4]), i32([0]), i32([0]))                      # rows of no sequence
    cache.compact(i32([0, 9, -1]), i32([-1, 0, 0]), i32([0, 0, 0, 0]), i32([0]))
    cache.compact(i32([0]), i32([4]), i32([0, 6]), i32([0, 1, 2, 3, 4, 5]))  # more than there are
    cache.compact(i32([0]), i32([4]), i32([0, 9]), i32([0]))                 # a range past keep
    same(cache, ref)


def test_append_rotates(attn):
    """k and q are turned as by rope(), bit for bit; v is not."""
    g = torch.Generator().manual_seed(8)
    cache, ref = make(attn, ps=16, D=64, H=2, max_pages=4, slots=3)
    new, seqs = [5, 0, 20], [2, 1, 0]
    start = cache.extend(i32(seqs), i32(new))
    ref.extend(seqs, new)
    qkv = torch.randn((25, 4 + 2 + 2, 64), generator=g).to(torch.bfloat16).to(DEV)
    q, k, v = qkv.split([4, 2, 2], 1)
    pos = i32([7, 1, 0, 30, 4] + list(range(20)))
    for rot, inter in ((64, False), (64, True), (20, False), (6, True)):
        tab = A.rope_table(range(31), rot).float().to(DEV)
        out = cache.append(k, v, i32([0, 5, 5, 25]), i32(seqs), start, layer=1, q=q, pos=pos, cos_sin=tab, interleaved=inter)
        assert torch.equal(out, attn.rope(q, pos, tab, interleaved=inter))
        kr = attn.rope(k, pos, tab, interleaved=inter)
        zero = torch.zeros((1, 25, 2, 64), dtype=torch.bfloat16)
        keep = ref.pool[0].clone()
        ref.append(torch.cat([zero, kr.cpu()[None]]), torch.cat([zero, v.cpu()[None]]), [0, 5, 5, 25], seqs, [0, 0, 0])
        ref.pool[0] = keep
        same(cache, ref)


def test_other_stream_and_graph(attn):
    """On a side stream, and replayed from a CUDA graph: the state moves with every replay."""
    cache, ref = make(attn)
    cache.extend(i32([0, 1]), i32([3, 4]))                # first calls load the kernels before the capture
    ref.extend([0, 1], [3, 4])
    k = torch.randn((2, 10, 2, 16), device=DEV).to(torch.bfloat16)
    seqs, new, cu = i32([1, 0]), i32([6, 4]), i32([0, 6, 10])
    cu_keep, keep = i32([0, 2, 4]), i32([0, 3, 1, 2])
    cache.append(k, k, cu, seqs, i32([-1, -1]), layer=None)
    cache.compact(seqs, i32([-1, -1]), cu_keep, keep)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        start = cache.extend(seqs, new)
        cache.append(k, k, cu, seqs, start, layer=None)
        cache.compact(seqs, start, cu_keep, keep)
    for _ in range(3):
        g.replay()
        s = ref.extend([1, 0], [6, 4])
        ref.append(k.cpu(), k.cpu(), [0, 6, 10], [1, 0], s)
        ref.compact([1, 0], s, [[0, 3], [1, 2]])
        assert start.tolist() == s
        same(cache, ref)


def test_offsets_past_32_bits(attn):
    """Pages behind 2^31 elements: layer and page offsets are 64-bit."""
    L, P, H, ps, D = 16, 1200, 8, 64, 128             # 1200 x 131072 = 1.6e8 elements a layer, 2.5e9 in all
    cache = attn.KVCache.create(L, P, ps, H, D, 2, 20, torch.bfloat16, DEV)
    cache.refs[:P - 4] = 1                            # only the last four pages are free
    start = cache.extend(i32([0]), i32([200]))
    assert start.tolist() == [0] and cache.table[0, :4].tolist() == [P - 4, P - 3, P - 2, P - 1]
    g = torch.Generator().manual_seed(1)
    k = torch.randn((L, 200, H, D), generator=g).to(torch.bfloat16).to(DEV)
    cache.append(k, k + 1, i32([0, 200]), i32([0]), start, layer=None)
    at = torch.arange(200, device=DEV)
    got = cache.pool[:, P - 4 + at // ps, :, :, at % ps]            # (200, L, 2, H, D)
    assert torch.equal(got[:, :, 0], k.transpose(0, 1)) and torch.equal(got[:, :, 1], (k + 1).transpose(0, 1))
    cache.compact(i32([0]), i32([100]), i32([0, 2]), i32([3, 99]))
    assert torch.equal(cache.pool[:, P - 4 + 101 // ps, 0, :, 101 % ps], k[:, 199])
    cache.copy(i32([P - 3]), i32([P - 1]))
    assert torch.equal(cache.pool[:, P - 1], cache.pool[:, P - 3])


def test_binding_refuses_wrong_tensors(attn):
    cache, _ = make(attn)
    k = torch.zeros((2, 2, 16), dtype=torch.bfloat16, device=DEV)
    ok = dict(cu=i32([0, 2]), seqs=i32([0]), start=i32([0]))
    for bad in (dict(k=k.float()), dict(k=k.cpu()), dict(k=k[:, :1]), dict(k=k, cu=i32([0])), dict(k=k, seqs=i32([0]).long()),
                dict(k=k, start=i32([0]).cpu()), dict(k=k, layer=None), dict(k=k.transpose(1, 2).contiguous().transpose(1, 2))):
        a = {**ok, **bad}
        with pytest.raises(AssertionError):
            cache.append(a["k"], a["k"], a["cu"], a["seqs"], a["start"], layer=a.get("layer", 0))
    with pytest.raises(AssertionError):
        cache.extend(i32([0]), i32([1, 2]))
    with pytest.raises(AssertionError):
        attn.attention(k.reshape(2, 2, 16), cache, i32([0, 2, 3]), i32([0]), i32([0]))
    from weight_only_int4_route_gb300 import moe
    with pytest.raises(moe.MoeError):
        cache.append(k, k, **ok, layer=2)
