"""The attention-side operators as measured workloads: rotary positions, the paged key/value cache,
attention of drafted tokens (trees) and of prompts over that cache.

Every case is run in two forms on the same inputs: `own` false computes it with elementary torch
operations in fp32, `own` true calls this package.  Layouts:

  pool   (layers, pages, 2, kv_heads, page_size, head_dim)  K at [:, :, 0], V at [:, :, 1]
  table  (slots, max_pages) int32, page of each page-sized piece of a sequence, -1 where there is none
  lens   (slots,) int32, tokens held;  refs (pages,) int32, sequences that hold a page (0 = free)
  cu     (n + 1,) int32, first row of each sequence's new tokens;  start (n,) int32, tokens held before them
  mask   (tokens, words) int32, bit j of row i: new token j of the same sequence is visible to it
  cos_sin (positions, rot) fp32, rot/2 cosines then rot/2 sines of a position
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases


def listed():
    return [
        # rotary ------------------------------------------------------------------------------
        # one decode step of 8 sequences: rotate q and k, put k and v into the cache
        dict(name="rope_decode", op="rope_append", dtype="bf16", n=8, new_lo=1, new_hi=1, ctx_lo=37, ctx_hi=900,
             q_heads=32, kv_heads=8, head_dim=128, rot=128, inter=False, page=16),
        # a prompt's queries inside their fused projection, interleaved pairs, half of the head rotated
        dict(name="rope_prompt", op="rope", dtype="f16", tokens=8192, heads=32, head_dim=128, rot=64, inter=True,
             inverse=False, pad=2048, positions=131072),
        # training: the gradient of rotated fp32 activations, an odd token count
        dict(name="rope_grad", op="rope", dtype="f32", tokens=40001, heads=16, head_dim=128, rot=128, inter=False,
             inverse=True, pad=0, positions=40960),
        # pages -------------------------------------------------------------------------------
        # a speculative step of 4 sequences on one layer: grow, write the draft, keep the accepted path, roll back
        dict(name="pages_step", op="step", dtype="bf16", layers=1, n=4, new_lo=5, new_hi=13, ctx_lo=60, ctx_hi=700,
             kv_heads=8, head_dim=128, page=16, keep_every=2),
        # the same on every layer of a model at once, a server's batch
        dict(name="pages_step_layers", op="step", dtype="bf16", layers=32, n=24, new_lo=9, new_hi=24, ctx_lo=100,
             ctx_hi=900, kv_heads=8, head_dim=128, page=32, keep_every=3),
        # parallel samples: fork, copy the shared last page when it is written, move pages, drop the samples
        dict(name="pages_fork", op="fork", dtype="bf16", layers=16, n=64, parents=8, ctx_lo=70, ctx_hi=1000,
             kv_heads=8, head_dim=128, page=64, moved=40),
        # drafted tokens over a cache ---------------------------------------------------------
        # one token of one sequence (latency)
        dict(name="tree_one", op="tree", dtype="bf16", n=1, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=1000, q_heads=16,
             kv_heads=16, head_dim=128, page=16),
        # trees of 8 to 32 drafted tokens, a server's batch of ragged contexts
        dict(name="tree_batch", op="tree", dtype="bf16", n=32, new_lo=8, new_hi=32, ctx_lo=500, ctx_hi=8000, q_heads=32,
             kv_heads=8, head_dim=128, page=64),
        # few sequences with long contexts: work has to be split along the keys
        dict(name="tree_long", op="tree", dtype="f16", n=5, new_lo=1, new_hi=60, ctx_lo=30000, ctx_hi=150000,
             q_heads=16, kv_heads=8, head_dim=64, page=32),
        # prompts -----------------------------------------------------------------------------
        # one short prompt
        dict(name="prompt_short", op="prompt", dtype="f16", n=1, new_lo=300, new_hi=300, ctx_lo=0, ctx_hi=0,
             q_heads=16, kv_heads=16, head_dim=64, page=16),
        # packed prompts of different lengths, some with a cached prefix
        dict(name="prompt_packed", op="prompt", dtype="bf16", n=6, new_lo=1, new_hi=2500, ctx_lo=0, ctx_hi=1500,
             q_heads=32, kv_heads=8, head_dim=128, page=64),
        # one long prompt (compute)
        dict(name="prompt_long", op="prompt", dtype="bf16", n=1, new_lo=8191, new_hi=8191, ctx_lo=0, ctx_hi=0,
             q_heads=32, kv_heads=8, head_dim=128, page=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope_append", "rope", "step", "fork", "tree", "tree", "tree", "prompt", "prompt"])
    dtype = rng.choice(["f16", "bf16"])
    head_dim = rng.choice([64, 128, 128, 80, 96])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        return dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), tokens=_log(rng, 1, 40000), heads=_log(rng, 1, 16),
                    head_dim=head_dim, rot=rng.choice([head_dim, head_dim // 2, 16]), inter=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 512]), positions=_log(rng, 256, 131072))
    if op == "rope_append":
        n, hi = _log(rng, 1, 64), _log(rng, 1, 300)
        return dict(op=op, dtype=dtype, n=n, new_lo=rng.randint(0, hi), new_hi=hi, ctx_lo=rng.randint(0, 50),
                    ctx_hi=_log(rng, 51, 2000), q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim,
                    rot=rng.choice([head_dim, head_dim // 2]), inter=rng.random() < 0.5, page=page)
    if op == "step":
        hi = _log(rng, 2, 40)
        return dict(op=op, dtype=dtype, layers=_log(rng, 1, 16), n=_log(rng, 1, 32), new_lo=rng.randint(0, hi),
                    new_hi=hi, ctx_lo=rng.randint(0, 60), ctx_hi=_log(rng, 61, 1000), kv_heads=kv_heads,
                    head_dim=head_dim, page=rng.choice([16, 32]), keep_every=rng.randint(1, 4))
    if op == "fork":
        n = _log(rng, 1, 64)
        return dict(op=op, dtype=dtype, layers=_log(rng, 1, 16), n=n, parents=rng.randint(1, n), ctx_lo=rng.randint(0, 60),
                    ctx_hi=_log(rng, 61, 800), kv_heads=kv_heads, head_dim=head_dim, page=rng.choice([16, 32, 64]),
                    moved=_log(rng, 1, 40))
    if op == "tree":
        n = _log(rng, 1, 32)
        ctx_hi = _log(rng, 64, min(100000, 200000 // n))
        hi = _log(rng, 1, 64)
        return dict(op=op, dtype=dtype, n=n, new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=rng.randint(0, ctx_hi),
                    ctx_hi=ctx_hi, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page)
    n = _log(rng, 1, 8)
    hi = _log(rng, 16, 6000 // n)
    ctx_hi = rng.choice([0, _log(rng, 1, 1500)])
    return dict(op="prompt", dtype=dtype, n=n, new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=rng.randint(0, ctx_hi),
                ctx_hi=ctx_hi, q_heads=kv_heads * min(group, 4), kv_heads=kv_heads, head_dim=head_dim, page=page)


def _spread(n, lo, hi, turn=0.6180339887):
    """n lengths over [lo, hi], the last one hi: the case alone fixes them, inputs vary by their values."""
    return [lo + round((hi - lo) * (((n - i) * turn) % 1.0)) for i in range(1, n)] + [hi]


def _lengths(c):
    return _spread(c["n"], c["new_lo"], c["new_hi"]), _spread(c["n"], c["ctx_lo"], c["ctx_hi"], 0.7548776662)


def _keep(c):
    """Accepted drafted tokens of each sequence: the first, then every keep_every-th."""
    return [list(range(0, m, c["keep_every"])) for m in _lengths(c)[0]]


def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rope":
        t = c["tokens"]
        return {"bytes": 2 * t * c["heads"] * c["head_dim"] * es + t * 4 + min(t, c["positions"]) * c["rot"] * 4,
                "flops": 3 * t * c["heads"] * c["rot"]}
    row = c["kv_heads"] * c["head_dim"] * es            # one token's K (or V) of one layer
    if c["op"] == "rope_append":
        t = sum(_lengths(c)[0])
        q = c["q_heads"] * c["head_dim"] * es
        return {"bytes": t * (2 * q + 4 * row + c["rot"] * 4), "flops": 3 * t * (c["q_heads"] + c["kv_heads"]) * c["rot"]}
    if c["op"] == "step":
        t = sum(_lengths(c)[0])
        moved = sum(1 for keep in _keep(c) for j, i in enumerate(keep) if i != j)
        return {"bytes": c["layers"] * row * 4 * (t + moved), "flops": 0}
    if c["op"] == "fork":
        partly = [x % c["page"] != 0 for x in _spread(c["parents"], c["ctx_lo"], c["ctx_hi"])]
        copied = sum(partly[i % c["parents"]] for i in range(c["n"])) + c["moved"]
        return {"bytes": copied * c["layers"] * c["page"] * row * 4, "flops": 0}
    new, ctx = _lengths(c)
    seen = sum(m * s + m * (m + 1) // 2 for m, s in zip(new, ctx))
    return {"bytes": sum(new) * c["q_heads"] * c["head_dim"] * es * 2 + sum(m + s for m, s in zip(new, ctx)) * row * 2,
            "flops": 4 * seen * c["q_heads"] * c["head_dim"]}


# ---------------------------------------------------------------- inputs


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(c, g, lens, slots, extra, max_len):
    """A cache whose sequences hold `lens` tokens on scattered pages; `extra` pages more than they need."""
    ps = c["page"]
    used = [-(-x // ps) for x in lens]
    pages = sum(used) + extra
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((slots, -(-max_len // ps)), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        refs[order[at:at + u].long()] = 1
        at += u
    pool = torch.randn((c.get("layers", 1), pages, 2, c["kv_heads"], ps, c["head_dim"]), generator=g, device=DEV,
                       dtype=torch.float32 if c["dtype"] == "f32" else DTYPES[c["dtype"]])
    full = torch.zeros(slots, dtype=torch.int32, device=DEV)
    full[:len(lens)] = _i32(lens)
    return dict(pool=pool, table=table, lens=full, refs=refs)


def _cos_sin(positions, rot, factor=4.0, base=10000.0):
    """Angles of positions compressed `factor` times for a long context, worked out in 64 bits."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot) / factor
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _tree_mask(r, new):
    """Random trees: each drafted token's parent is an earlier one or the context; rows see themselves and their ancestors."""
    words = -(-max(new) // 32)
    rows = []
    for m in new:
        own_bits = []
        for i in range(m):
            p = r.randrange(-1, i)
            own_bits.append((own_bits[p] if p >= 0 else 0) | (1 << i))
        rows += own_bits
    return torch.tensor([[(b >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for b in rows], dtype=torch.int64,
                        device=DEV).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = random.Random(seed)
    dt = DTYPES[c["dtype"]]
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=dt)  # noqa: E731
    if c["op"] == "rope":
        t, width = c["tokens"], c["heads"] * c["head_dim"]
        x = randn(t, width + c["pad"])[:, :width].unflatten(1, (c["heads"], c["head_dim"]))
        pos = torch.randint(0, c["positions"], (t,), generator=g, device=DEV).to(torch.int32)
        return dict(case=c, x=x, pos=pos, cos_sin=_cos_sin(c["positions"], c["rot"]))
    if c["op"] == "fork":
        lens = _spread(c["parents"], c["ctx_lo"], c["ctx_hi"])
        s = _cache(c, g, lens, c["parents"] + c["n"], c["n"] * 2 + 2 * c["moved"], c["ctx_hi"] + 1)
        free = (s["refs"] == 0).nonzero().flatten().to(torch.int32)
        held = (s["refs"] > 0).nonzero().flatten().to(torch.int32)
        pick = torch.randint(0, held.numel(), (c["moved"],), generator=g, device=DEV)
        return dict(case=c, **s, src=_i32([i % c["parents"] for i in range(c["n"])]),
                    dst=_i32([c["parents"] + i for i in range(c["n"])]), one=torch.ones(c["n"], dtype=torch.int32, device=DEV),
                    copy_src=held[pick].contiguous(), copy_dst=free[-c["moved"]:].flip(0).contiguous())
    new, ctx = _lengths(c)
    t = sum(new)
    seqs = list(range(c["n"]))
    r.shuffle(seqs)
    at = [0] * c["n"]
    for i, q in enumerate(seqs):
        at[q] = i                               # slot q holds the i-th sequence of the batch
    cu = _i32([sum(new[:i]) for i in range(c["n"] + 1)])
    most = max(m + s for m, s in zip(new, ctx))
    if c["op"] == "step":
        s = _cache(c, g, [ctx[at[q]] for q in range(c["n"])], c["n"], sum(-(-m // c["page"]) + 1 for m in new), most)
        keep = _keep(c)
        return dict(case=c, **s, seqs=_i32(seqs), new=_i32(new), cu=cu, k=randn(c["layers"], t, c["kv_heads"], c["head_dim"]),
                    v=randn(c["layers"], t, c["kv_heads"], c["head_dim"]),
                    keep=_i32([i for x in keep for i in x]), cu_keep=_i32([sum(map(len, keep[:i])) for i in range(c["n"] + 1)]),
                    none=torch.zeros(c["n"] + 1, dtype=torch.int32, device=DEV))
    held = [new[at[q]] + ctx[at[q]] for q in range(c["n"])]
    s = _cache(c, g, held, c["n"], 7, most)
    base = dict(case=c, **s, seqs=_i32(seqs), start=_i32(ctx), cu=cu)
    if c["op"] == "rope_append":
        width = (c["q_heads"] + 2 * c["kv_heads"]) * c["head_dim"]
        qkv = randn(t, width).unflatten(1, (-1, c["head_dim"]))     # the fused projection's output
        pos = torch.cat([_i32(range(s, s + m)) for m, s in zip(new, ctx)])
        return dict(base, qkv=qkv, pos=pos, cos_sin=_cos_sin(most + 1, c["rot"]))
    q = randn(t, c["q_heads"], c["head_dim"]) * 2
    return dict(base, q=q, mask=_tree_mask(r, new) if c["op"] == "tree" else None)


# ---------------------------------------------------------------- the package's form


def _own(s):
    from weight_only_int4_route_gb300 import attn
    c = s["case"]
    if c["op"] == "rope":
        return attn.rope(s["x"], s["pos"], s["cos_sin"], interleaved=c["inter"], inverse=c["inverse"])
    cache = attn.KVCache(s["pool"], s["table"], s["lens"], s["refs"])
    if c["op"] == "rope_append":
        q, k, v = s["qkv"].split([c["q_heads"], c["kv_heads"], c["kv_heads"]], 1)
        q = cache.append(k, v, s["cu"], s["seqs"], s["start"], q=q, pos=s["pos"], cos_sin=s["cos_sin"], interleaved=c["inter"])
        return {"q": q, "pool": s["pool"]}
    if c["op"] == "step":
        start = cache.extend(s["seqs"], s["new"])
        cache.append(s["k"], s["v"], s["cu"], s["seqs"], start, layer=None)
        cache.compact(s["seqs"], start, s["cu_keep"], s["keep"])
        table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
        cache.compact(s["seqs"], start, s["none"], s["keep"])
        return {"start": start, "table": table, "lens": lens, "refs": refs, "pool": s["pool"], "free": s["refs"]}
    if c["op"] == "fork":
        cache.fork(s["src"], s["dst"])
        start = cache.extend(s["dst"], s["one"])
        cache.copy(s["copy_src"], s["copy_dst"])
        table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
        cache.free(s["dst"])
        return {"start": start, "table": table, "lens": lens, "refs": refs, "pool": s["pool"], "free": s["refs"]}
    out, lse = attn.attention(s["q"], cache, s["cu"], s["seqs"], s["start"], mask=s["mask"], return_lse=True)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- plain forms


def _rotate(x, pos, cos_sin, inter, inverse, dtype=torch.float32):
    rot = cos_sin.shape[1]
    cos, sin = cos_sin.to(dtype)[pos.long(), None].chunk(2, 2)
    sin = -sin if inverse else sin
    y = x.to(dtype)
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _rows(s, count, start):
    """Pages and slots of the new tokens: (page, slot) of each row."""
    t = int(count.sum())
    of = torch.repeat_interleave(torch.arange(count.numel(), device=DEV), count.long())
    at = start.long()[of] + torch.arange(t, device=DEV) - (count.cumsum(0) - count).long()[of]
    ps = s["pool"].shape[4]
    return s["table"][s["seqs"].long()[of], at // ps].long(), at % ps


def _extend(s, seqs, new):
    """Grow sequences: the lowest free pages in order; a partly filled last page that others hold too is copied."""
    pool, table, lens, refs = s["pool"], s["table"], s["lens"], s["refs"]
    ps, q = pool.shape[4], seqs.long()
    old = lens[q].long()
    have, want = (old + ps - 1) // ps, (old + new + ps - 1) // ps
    last = table[q, (old // ps).clamp(max=table.shape[1] - 1)].long()
    part = (old % ps > 0) & (new > 0)
    cow = part & (refs[last.clamp(min=0)] > 1)
    need = want - have + cow
    total = int(need.sum())
    page = (refs == 0).nonzero().flatten()[:total]
    if page.numel() < total or int(want.max()) > table.shape[1]:
        return torch.full_like(seqs, -1)
    of = torch.repeat_interleave(torch.arange(q.numel(), device=DEV), need)
    nth = torch.arange(total, device=DEV) - (need.cumsum(0) - need)[of]
    first = torch.where(cow, old // ps, have)
    table[q[of], first[of] + nth] = page.to(torch.int32)
    refs[page] = 1
    copies = cow[of] & (nth == 0)
    pool[:, page[copies]] = pool[:, last[of][copies]]
    refs.index_add_(0, last[cow], torch.full_like(last[cow], -1).to(torch.int32))
    lens[q] = (old + new).to(torch.int32)
    return old.to(torch.int32)


def _drop(s, q, first, end):
    """Release the pages [first, end) of the tables' rows q."""
    col = torch.arange(s["table"].shape[1], device=DEV)
    gone = (col >= first[:, None]) & (col < end[:, None])
    rows = s["table"][q]
    pages = rows[gone].long()
    s["refs"].index_add_(0, pages, torch.full_like(pages, -1).to(torch.int32))
    s["table"][q] = torch.where(gone, -1, rows)


def _compact(s, seqs, start, cu_keep, keep):
    pool, q, ps = s["pool"], seqs.long(), s["pool"].shape[4]
    count = cu_keep.diff().long()
    of = torch.repeat_interleave(torch.arange(q.numel(), device=DEV), count)
    nth = torch.arange(of.numel(), device=DEV) - (count.cumsum(0) - count)[of]
    src, dst = start.long()[of] + keep.long()[:of.numel()], start.long()[of] + nth
    rows = s["table"][q][of].long()
    pick = lambda at: rows.gather(1, (at // ps)[:, None])[:, 0]  # noqa: E731
    pool[:, pick(dst), :, :, dst % ps] = pool[:, pick(src), :, :, src % ps]
    end = (s["lens"][q].long() + ps - 1) // ps
    s["lens"][q] = (start.long() + count).to(torch.int32)
    _drop(s, q, (start.long() + count + ps - 1) // ps, end)


def _attend(s, dtype=torch.float32):
    """softmax(q k^T / sqrt(head_dim)) v over the visible keys, all sequences padded to the longest; (out, lse)."""
    c, q, pool = s["case"], s["q"], s["pool"][0]
    hk, ps, d = pool.shape[2:]
    grp = q.shape[1] // hk
    count = s["cu"].diff().long()
    held = s["start"].long() + count
    nq, nk = int(count.max()), int(held.max())
    pages = s["table"][s["seqs"].long(), :-(-nk // ps)].long().clamp(min=0)
    key = torch.arange(nk, device=DEV)
    there = (key < held[:, None])[:, None, :, None]
    k, v = (torch.where(there, pool[pages, i].transpose(1, 2).flatten(2, 3)[:, :, :nk], 0).to(dtype) for i in (0, 1))
    i = torch.arange(nq, device=DEV)
    row = (s["cu"][:-1, None].long() + i).clamp(max=q.shape[0] - 1)
    x = q[row].to(dtype).unflatten(2, (hk, grp)).permute(0, 2, 3, 1, 4).flatten(2, 3)     # n, hk, grp * nq, d
    rel = key - s["start"].long()[:, None, None]
    if s["mask"] is None:
        see = rel <= i[:, None]
    else:
        words = s["mask"][row].long()
        j = rel.clamp(0, words.shape[2] * 32 - 1).expand(-1, nq, -1)
        see = ((words.gather(2, j // 32) >> (j % 32)) & 1).bool() | ((rel < 0) & (words != 0).any(2, keepdim=True))
    see = (see & (key < held[:, None, None]))[:, None, None]
    score = (x @ k.transpose(2, 3)).div_(math.sqrt(d)).unflatten(2, (grp, nq)).masked_fill_(~see, -math.inf)
    top = score.amax(4, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    p = score.sub_(top).exp_()
    total = p.sum(4, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (grp, nq)) / torch.where(total == 0, 1, total)
    lse = (total.log() + top)[..., 0]
    ok = i < count[:, None]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[ok]
    return o, lse.permute(0, 3, 1, 2).flatten(2, 3)[ok]


def run(s):
    if own:
        return _own(s)
    c = s["case"]
    if c["op"] == "rope":
        return _rotate(s["x"], s["pos"], s["cos_sin"], c["inter"], c["inverse"]).to(s["x"].dtype)
    if c["op"] == "rope_append":
        q, k, v = s["qkv"].split([c["q_heads"], c["kv_heads"], c["kv_heads"]], 1)
        page, slot = _rows(s, s["cu"].diff(), s["start"])
        s["pool"][0, page, 0, :, slot] = _rotate(k, s["pos"], s["cos_sin"], c["inter"], False).to(k.dtype)
        s["pool"][0, page, 1, :, slot] = v
        return {"q": _rotate(q, s["pos"], s["cos_sin"], c["inter"], False).to(q.dtype), "pool": s["pool"]}
    if c["op"] == "step":
        start = _extend(s, s["seqs"], s["new"])
        page, slot = _rows(s, s["cu"].diff(), start)
        s["pool"][:, page, 0, :, slot] = s["k"].transpose(0, 1)
        s["pool"][:, page, 1, :, slot] = s["v"].transpose(0, 1)
        _compact(s, s["seqs"], start, s["cu_keep"], s["keep"])
        table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
        _compact(s, s["seqs"], start, s["none"], s["keep"])
        return {"start": start, "table": table, "lens": lens, "refs": refs, "pool": s["pool"], "free": s["refs"]}
    if c["op"] == "fork":
        src, dst = s["src"].long(), s["dst"].long()
        s["table"][dst], s["lens"][dst] = s["table"][src], s["lens"][src]
        pages = s["table"][src]
        pages = pages[pages >= 0].long()
        s["refs"].index_add_(0, pages, torch.ones_like(pages).to(torch.int32))
        start = _extend(s, s["dst"], s["one"])
        s["pool"][:, s["copy_dst"].long()] = s["pool"][:, s["copy_src"].long()]
        table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
        _drop(s, dst, torch.zeros_like(dst), (s["lens"][dst].long() + c["page"] - 1) // c["page"])
        s["lens"][dst] = 0
        return {"start": start, "table": table, "lens": lens, "refs": refs, "pool": s["pool"], "free": s["refs"]}
    out, lse = _attend(s)
    return {"out": out.to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] in ("step", "fork"):
        return None                             # values are moved, not computed
    if c["op"] in ("rope", "rope_append"):
        rot = c["rot"]
        ang = s["cos_sin"].double()[s["pos"].long()]
        w = torch.complex(ang[:, :rot // 2], ang[:, rot // 2:])
        w = (w.conj() if c.get("inverse") else w)[:, None]

        def turn(x):                            # the pairs of a head as complex numbers, times the position's
            x = x.double()
            lo = torch.arange(0, rot, 2, device=DEV) if c["inter"] else torch.arange(rot // 2, device=DEV)
            hi = lo + 1 if c["inter"] else lo + rot // 2
            y, z = x.clone(), torch.complex(x[..., lo], x[..., hi]) * w
            y[..., lo], y[..., hi] = z.real, z.imag
            return y

        if c["op"] == "rope":
            return turn(s["x"])
        hq, hk = c["q_heads"], c["kv_heads"]
        pool = s["pool"].double()
        k, v = turn(s["qkv"][:, hq:hq + hk]), s["qkv"][:, hq + hk:].double()
        cu, start, seqs = s["cu"].tolist(), s["start"].tolist(), s["seqs"].tolist()
        for b in range(c["n"]):
            at = start[b] + torch.arange(cu[b + 1] - cu[b], device=DEV)
            page = s["table"][seqs[b]].long()[at // c["page"]]
            pool[0, page, 0, :, at % c["page"]] = k[cu[b]:cu[b + 1]]
            pool[0, page, 1, :, at % c["page"]] = v[cu[b]:cu[b + 1]]
        return {"q": turn(s["qkv"][:, :hq]), "pool": pool}
    cu, start, seqs = s["cu"].tolist(), s["start"].tolist(), s["seqs"].tolist()
    d, hk, hq = c["head_dim"], c["kv_heads"], c["q_heads"]
    out = torch.zeros((cu[-1], hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((cu[-1], hq), dtype=torch.float64, device=DEV)
    for b in range(c["n"]):
        m, n0 = cu[b + 1] - cu[b], start[b]
        n = m + n0
        pages = s["table"][seqs[b], :-(-n // c["page"])].long()
        see = torch.ones((m, n), dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            see[:, n0:] = torch.ones((m, m), dtype=torch.bool, device=DEV).tril()
        else:
            bits = s["mask"][cu[b]:cu[b + 1]].long()[:, :, None] >> torch.arange(32, device=DEV)
            see[:, n0:] = (bits & 1).flatten(1)[:, :m].bool()
        for h in range(hk):
            k, v = (s["pool"][0, pages, i, h].flatten(0, 1)[:n].double() for i in (0, 1))
            for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                score = (s["q"][cu[b]:cu[b + 1], g].double() @ k.T / math.sqrt(d)).masked_fill(~see, -math.inf)
                lse[cu[b]:cu[b + 1], g] = score.logsumexp(1)
                out[cu[b]:cu[b + 1], g] = score.softmax(1) @ v
    return {"out": out, "lse": lse}
