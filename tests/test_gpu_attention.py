"""Attention over the paged cache on the GPU against the float64 oracle.

Bounds, elementwise, with u the type's unit roundoff (2^-8 bf16, 2^-11 f16), A = sum_j p_j |v_j| and S = the
largest sum_d scale |q_d k_d| of the row.  A score is a head_dim-term fp32 dot product, its terms added on the tensor
cores with at worst truncated additions: off by at most 2^-18 S for head_dim <= 128 (128 additions of 2^-23, twice for
safety), a weight by a factor of at most e^(2^-17 S) after the division by the sum, which carries the same errors.
The weights are rounded to the type for their product with V (u A), the sums are fp32 (2^-16 A covers 2^15 keys per running
sum), and the output is rounded once (u |out|).  f16 weights below 2^-24 of the scaled range vanish: with the range used
(weights up to 2^15) they are below 2^-30 of the largest, n of them below n 2^-30 max|v|."""
import math
import random

import pytest
import torch

from _helpers import have_gpu
from oracle import attn_oracle as A

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a CUDA GPU")]
DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
B16, H16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def attn():
    from weight_only_int4_route_gb300 import attn, build, moe
    build.build()
    moe.lib()
    yield attn
    assert moe.device_error(DEV) == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Case:
    """Sequences of ctx + new tokens on scattered pages of a pool that holds NaN everywhere else."""

    def __init__(self, attn, dtype, Hq, Hk, D, ps, new, ctx, seed=0, layers=1, layer=0, spread=2.0):
        g = torch.Generator().manual_seed(seed)
        r = random.Random(seed)
        self.attn, self.D, self.new, self.ctx, self.dtype, self.layer, self.Hk = attn, D, new, ctx, dtype, layer, Hk
        n = len(new)
        need = [-(-(a + b) // ps) for a, b in zip(new, ctx)]
        pages = sum(need) + 3
        order = list(range(pages))
        r.shuffle(order)
        self.slots = list(range(n + 1))
        r.shuffle(self.slots)
        self.slots = self.slots[:n]
        pool = torch.full((layers, pages, 2, Hk, ps, D), math.nan, dtype=dtype)
        table = torch.full((n + 1, max(need + [1])), -1, dtype=torch.int32)
        self.k, self.v = [], []
        at = 0
        for b in range(n):
            m = new[b] + ctx[b]
            k, v = (torch.randn((Hk, m, D), generator=g).to(dtype) for _ in range(2))
            self.k.append(k)
            self.v.append(v)
            for i in range(need[b]):
                p = order[at]
                at += 1
                table[self.slots[b], i] = p
                c = min(ps, m - i * ps)
                pool[layer, p, 0, :, :c], pool[layer, p, 1, :, :c] = k[:, i * ps:i * ps + c], v[:, i * ps:i * ps + c]
        T = sum(new)
        self.q = (torch.randn((T, Hq, D), generator=g) * spread).to(dtype)
        self.cu = [sum(new[:i]) for i in range(n + 1)]
        lens, refs = torch.zeros(n + 1, dtype=torch.int32), torch.zeros(pages, dtype=torch.int32)
        self.cache = attn.KVCache(pool.to(DEV), table.to(DEV), lens.to(DEV), refs.to(DEV))
        self.see = [[range(s + i + 1) for i in range(m)] for m, s in zip(new, ctx)]
        self.mask = None

    def with_sets(self, sets, words):
        """sets: per row the visible drafted tokens (none at all: padding)."""
        self.mask = A.bits(sets, words).to(DEV)
        self.see = []
        for b, (m, s) in enumerate(zip(self.new, self.ctx)):
            rows = sets[self.cu[b]:self.cu[b + 1]]
            self.see.append([list(range(s)) + [s + j for j in sorted(x) if j < min(m, 32 * words)] if x else [] for x in rows])
        return self

    def run(self, q=None, **kw):
        return self.attn.attention(self.q.to(DEV) if q is None else q, self.cache, i32(self.cu), i32(self.slots),
                                   i32(self.ctx), mask=self.mask, layer=self.layer, return_lse=True, **kw)

    def check(self, out, lse, scale=None):
        out, lse = out.double().cpu(), lse.double().cpu()
        u = U[self.dtype]
        for b in range(len(self.new)):
            rows = slice(self.cu[b], self.cu[b + 1])
            ref, ref_lse, mag, s = A.attention(self.q[rows], self.k[b], self.v[b], self.see[b], scale or self.D ** -0.5)
            empty = ref_lse == -math.inf
            assert (lse[rows][empty] == -math.inf).all() and not out[rows][empty].any(), "rows that see nothing"
            if not ref.numel():
                continue
            n = self.k[b].shape[1]
            vmax = float(self.v[b].double().abs().nan_to_num(0, 0, 0).max()) if n else 0.0
            e = (2.0 ** -17 * s).clamp(max=0.5)
            bound = (u * (1 + 2 ** -6) + 3 * e + 2.0 ** -16)[..., None] * mag + u * ref.abs() + n * 2.0 ** -30 * vmax + 1e-30
            off = (out[rows] - ref).abs()
            assert not (off > bound).any() and torch.isfinite(out[rows]).all(), (b, float((off / bound).max()))
            good = ~empty
            lo = (lse[rows] - ref_lse)[good].abs()
            assert not (lo > (e + 2.0 ** -16 + 2.0 ** -22 * ref_lse.abs())[good]).any(), (b, float(lo.max()))


CAUSAL = [
    # dtype, Hq, Hk, D, page, new, ctx
    (B16, 1, 1, 8, 8, [1], [0]),
    (B16, 4, 1, 64, 16, [1], [0]),
    (H16, 4, 4, 64, 16, [1, 1, 1], [0, 1, 129]),
    (B16, 8, 2, 128, 16, [5, 0, 1, 17], [0, 33, 127, 128]),
    (H16, 6, 2, 80, 32, [3, 40], [255, 256]),
    (B16, 5, 1, 96, 64, [130], [70]),
    (B16, 2, 2, 128, 128, [257], [0]),
    (H16, 3, 3, 64, 256, [127, 128, 129], [1, 0, 300]),
    (B16, 128, 1, 64, 16, [3], [40]),
    (H16, 7, 1, 72, 8, [20, 1], [9, 700]),
    (B16, 12, 4, 40, 16, [64, 65, 1, 0, 2], [64, 63, 1000, 5, 0]),
    (H16, 32, 8, 128, 64, [1] * 9, [1, 64, 127, 128, 129, 500, 0, 1023, 64]),
    (B16, 4, 2, 24, 8, [300], [1]),
    (B16, 2, 1, 128, 16, [1], [9000]),
    (H16, 16, 2, 128, 32, [9, 1], [5000, 3]),
    (B16, 8, 8, 128, 64, [1500], [0]),       # several items and several key tiles per block
    (H16, 8, 8, 64, 16, [1100, 700, 0, 300], [130, 0, 7, 1000]),
    (B16, 6, 2, 64, 32, [1100, 300, 85], [70, 0, 3]),        # groups that do not divide a tile of rows
    (H16, 10, 2, 96, 8, [500, 26, 600], [5, 400, 127]),
    (B16, 14, 2, 128, 64, [37, 400], [1000, 333]),
]


@pytest.mark.parametrize("i", range(len(CAUSAL)))
def test_causal(attn, i):
    c = Case(attn, *CAUSAL[i], seed=i)
    c.check(*c.run())


@pytest.mark.parametrize("i", range(len(CAUSAL)))
def test_masked(attn, i):
    """Random bits, rows without any among them; words for all, for too few and for more than the tokens."""
    c = Case(attn, *CAUSAL[i], seed=100 + i)
    r = random.Random(i)
    most = max(c.new)
    words = max(1, [-(-most // 32), most // 32, most // 32 + 2][i % 3])
    sets = []
    for m in c.new:
        for j in range(m):
            n = r.choice([0, 1, 1, m // 2, m])
            sets.append({x for x in r.sample(range(m), min(n, m)) if x < 32 * words})
    c.with_sets(sets, words)
    c.check(*c.run())


@pytest.mark.parametrize("dtype,G,D", [(B16, 1, 128), (H16, 4, 64), (B16, 8, 128)])
def test_trees(attn, dtype, G, D):
    """tree_mask's bits and positions, and the attention of the trees."""
    r = random.Random(G)
    new, ctx = [1, 12, 33, 64, 2, 90], [0, 500, 3, 131, 1, 2000]
    c = Case(attn, dtype, 2 * G, 2, D, 16, new, ctx, seed=G)
    parents = [r.choice([-1, r.randint(-1, i - 1), i - 1, -2 if r.random() < 0.1 else i - 1]) if i else -1
               for m in new for i in range(m)]
    for limit in (90, 64):
        words = -(-limit // 32)
        sets, pos = A.tree_mask(parents, c.cu, ctx, words)
        mask, got = attn.tree_mask(i32(parents), i32(c.cu), i32(ctx), limit)
        assert got.tolist() == pos and torch.equal(mask.cpu(), A.bits(sets, words))
        c.with_sets(sets, words)
        c.check(*c.run())


def test_a_chain_is_causal(attn):
    new, ctx = [40, 3], [77, 200]
    c = Case(attn, B16, 8, 2, 128, 16, new, ctx, seed=5)
    out, lse = c.run()
    c.mask, _ = attn.tree_mask(i32([i - 1 for m in new for i in range(m)]), i32(c.cu), i32(ctx), 40)
    out2, lse2 = c.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_unseen_values_have_no_influence(attn, bad):
    """A drafted token holding NaN or infinities in K and V changes only the rows that see it."""
    new, ctx = [30], [100]
    c = Case(attn, B16, 4, 2, 64, 16, new, ctx, seed=6)
    sets = [({j for j in range(i + 1)} - {7} if i != 20 else {7, 20}) for i in range(30)]
    sets[7] = {3}
    c.with_sets(sets, 1)
    clean, clean_lse = c.run()
    p, x = int(c.cache.table[c.slots[0], 107 // 16]), 107 % 16
    c.cache.pool[0, p, 0, :, x] = bad
    c.cache.pool[0, p, 1, :, x] = bad
    out, lse = c.run()
    rest = [i for i in range(30) if i != 20]
    c.see[0][20] = []
    assert not torch.isfinite(out[20]).all()
    out[20], lse[20] = 0, -math.inf
    c.check(out, lse)
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
    # V alone: rows that see it carry it through, the others do not
    c.cache.pool[0, p, 0, :, x] = c.k[0][:, 107].to(DEV)
    out, lse = c.run()
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse, clean_lse)
    assert (torch.isnan(out[20]) if bad != bad else out[20] == bad).all()


def test_causal_rows_before_a_bad_token(attn):
    c = Case(attn, H16, 2, 1, 128, 16, [200], [10], seed=7)
    clean, _ = c.run()
    pos = 10 + 90
    p = int(c.cache.table[c.slots[0], pos // 16])
    c.cache.pool[0, p, 1, :, pos % 16, 5] = math.inf
    c.cache.pool[0, p, 1, :, pos % 16, 70] = math.nan
    out, _ = c.run()
    assert torch.equal(out[:90], clean[:90])
    keep = [d for d in range(128) if d not in (5, 70)]
    assert torch.equal(out[90:][..., keep], clean[90:][..., keep])
    assert (out[90:, :, 5] == math.inf).all() and torch.isnan(out[90:, :, 70]).all()


@pytest.mark.parametrize("dtype,Hq,Hk,D,new,ctx", [(B16, 4, 2, 128, [700, 90], [60, 300]), (H16, 2, 2, 64, [900], [0]),
                                                   (B16, 8, 1, 64, [25, 3], [4000, 2000])])
def test_bad_tokens_reach_only_later_rows(attn, dtype, Hq, Hk, D, new, ctx):
    """V elements that are not finite, in several tiles, pieces and both row tiles of an item: a causal row is touched where it
    sees one, and nowhere else."""
    c = Case(attn, dtype, Hq, Hk, D, 16, new, ctx, seed=21)
    clean, lse0 = c.run()
    r = random.Random(4)
    hit = {}
    for b in range(len(new)):
        for at in sorted(r.sample(range(new[b]), 2)):
            d, h, bad = r.randrange(D), r.randrange(Hk), r.choice([math.nan, math.inf, -math.inf])
            pos = ctx[b] + at
            p = int(c.cache.table[c.slots[b], pos // 16])
            c.cache.pool[0, p, 1, h, pos % 16, d] = bad
            hit.setdefault((b, h, d), []).append((at, bad))
    out, lse = c.run()
    assert torch.equal(lse, lse0)
    want = clean.clone()
    grp = Hq // Hk
    for (b, h, d), bads in hit.items():
        for at, bad in bads:
            want[c.cu[b] + at:c.cu[b + 1], h * grp:(h + 1) * grp, d] += bad
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(nan=0.0, posinf=1e4, neginf=-1e4), want.nan_to_num(nan=0.0, posinf=1e4, neginf=-1e4))


def test_bad_context_reaches_every_row_but_padding(attn):
    c = Case(attn, B16, 2, 1, 64, 16, [4], [300], seed=22)
    c.with_sets([{0}, set(), {0, 2}, {3}], 1)
    clean, _ = c.run()
    p = int(c.cache.table[c.slots[0], 9])
    c.cache.pool[0, p, 1, 0, 3, 7] = math.nan
    out, lse = c.run()
    assert torch.isnan(out[[0, 2, 3], :, 7]).all() and not out[1].any() and (lse[1] == -math.inf).all()
    keep = [d for d in range(64) if d != 7]
    assert torch.equal(out[..., keep], clean[..., keep])


def test_extreme_values(attn):
    """f16 values near the type's largest, all weights alike: the sum of weights is kept in range."""
    c = Case(attn, H16, 2, 1, 64, 16, [3], [1000], seed=23, spread=0.0)
    for i in range(c.cache.table.shape[1]):
        p = int(c.cache.table[c.slots[0], i])
        n = min(16, 1003 - 16 * i)
        c.v[0][:, 16 * i:16 * i + n] = 60000.0
        c.cache.pool[0, p, 1, :, :n] = 60000.0
    c.check(*c.run())


def test_one_token_of_any_stride(attn):
    """torch leaves the stride of a dimension of one open."""
    c = Case(attn, B16, 4, 2, 64, 16, [1], [50], seed=24)
    out, _ = c.run()
    odd = torch.empty(4 * 64 + 8, dtype=B16, device=DEV)[:256].as_strided((1, 4, 64), (3, 64, 1))
    odd.copy_(c.q.to(DEV))
    assert torch.equal(c.run(q=odd)[0], out)


def test_large_scores(attn):
    """Scores far apart: a running maximum that grows from tile to tile, weights that underflow."""
    c = Case(attn, B16, 4, 1, 64, 16, [6], [700], seed=8, spread=1.0)
    ramp = torch.linspace(0.1, 12.0, 706)
    k = (c.k[0].float().sign() * ramp[None, :, None]).to(B16)
    c.k[0] = k
    for i in range(c.cache.table.shape[1]):
        p = int(c.cache.table[c.slots[0], i])
        n = min(16, 706 - 16 * i)
        c.cache.pool[0, p, 0, :, :n] = k[:, 16 * i:16 * i + n].to(DEV)
    for scale in (0.125, 1.0, 4.0):
        c.check(*c.run(scale=scale), scale=scale)


def test_skipped_sequences_and_layers(attn):
    """A negative start or a slot that does not exist sees nothing; other layers are not touched."""
    c = Case(attn, B16, 4, 2, 64, 16, [3, 4, 5], [20, 30, 40], seed=9, layers=3, layer=2)
    out, lse = c.run()
    c.check(out, lse)
    out2, lse2 = attn.attention(c.q.to(DEV), c.cache, i32(c.cu), i32([c.slots[0], 77, c.slots[2]]), i32([20, 30, -1]),
                                layer=2, return_lse=True)
    assert torch.equal(out2[:3], out[:3]) and not out2[3:].any() and (lse2[3:] == -math.inf).all()


def test_strided_queries_rows_of_no_sequence_and_no_lse(attn):
    c = Case(attn, B16, 8, 2, 64, 16, [9, 20], [50, 0], seed=10)
    out, lse = c.run()
    wide = torch.zeros((29, 12, 64), dtype=B16, device=DEV)
    wide[:, 2:10] = c.q.to(DEV)
    out2, lse2 = c.run(q=wide[:, 2:10])
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    part = attn.attention(c.q.to(DEV), c.cache, i32([9, 29]), i32(c.slots[1:]), i32(c.ctx[1:]))
    assert torch.equal(part[9:], out[9:])


def test_runs_agree_and_other_streams(attn):
    """The same bits on every run, whatever the workspace held, on another stream and from a graph."""
    c = Case(attn, H16, 16, 4, 128, 32, [1, 9, 33], [7000, 100, 2500], seed=11)
    out, lse = c.run()
    junk = torch.full((200 << 20,), 0xFF, dtype=torch.uint8, device=DEV)      # the next workspaces hold NaN
    torch.cuda.synchronize()
    del junk
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, cu, seqs, start = c.q.to(DEV), i32(c.cu), i32(c.slots), i32(c.ctx)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            o, s = attn.attention(q, c.cache, cu, seqs, start, return_lse=True)
            side.synchronize()
            assert torch.equal(o, out) and torch.equal(s, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, s = attn.attention(q, c.cache, cu, seqs, start, return_lse=True)
    for _ in range(2):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(s, lse)


def test_many_sequences(attn):
    """More sequences than a block has threads, lengths from nothing on."""
    n = 700
    r = random.Random(3)
    c = Case(attn, B16, 2, 1, 16, 8, [r.choice([0, 1, 1, 1, 2, 5]) for _ in range(n)], [r.randint(0, 40) for _ in range(n)], seed=12)
    c.check(*c.run())


def test_many_prompts(attn):
    """More prompts than a block has threads, each of several rows tiles."""
    n = 300
    r = random.Random(5)
    c = Case(attn, H16, 4, 1, 16, 16, [r.choice([40, 70, 33, 1]) for _ in range(n)], [r.randint(0, 60) for _ in range(n)], seed=15)
    c.check(*c.run())


def test_offsets_past_32_bits(attn):
    """The sequence's pages lie behind 2^32 bytes and 2^31 elements of the pool."""
    P, Hk, ps, D = 20000, 8, 64, 128                       # 2.6e9 elements
    pool = torch.zeros((1, P, 2, Hk, ps, D), dtype=B16, device=DEV)
    c = Case(attn, B16, 8, 8, D, ps, [3], [250], seed=13)
    used = c.cache.table[c.slots[0], :4].tolist()
    table = c.cache.table.clone()
    for i, p in enumerate(used):
        pool[0, P - 1 - i] = c.cache.pool[0, p]
        table[c.slots[0], i] = P - 1 - i
    c.cache = attn.KVCache(pool, table, c.cache.lens, torch.zeros(P, dtype=torch.int32, device=DEV))
    c.check(*c.run())


def test_long_context(attn):
    """One token over 100,000 cached ones: split along the keys and joined."""
    c = Case(attn, H16, 4, 1, 64, 128, [1], [100001], seed=14, spread=1.0)
    c.check(*c.run())
