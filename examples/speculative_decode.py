"""A small decoder that drafts and verifies trees of tokens: the attention operators beside the expert layer.

Every layer is attention over the paged cache (rotary positions, cache write, grouped heads) followed by the quantized
expert layer.  A prompt goes through causally; then each round drafts a tree of tokens, verifies it in one pass, keeps the
longest path the model itself would have taken and drops the rest of the draft from the cache.  The routed experts of the
draft are counted in the expert lookahead buffer.  Weights are random, so the draft comes from the model's own ranking of
the last verified token; what matters is the flow.

    python examples/speculative_decode.py [rounds]
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_only_int4_route_gb300 import attn, moe, synth  # noqa: E402

DEV = "cuda:0"


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Decoder:
    def __init__(self, cfg, layers=2, q_heads=4, kv_heads=2, head_dim=64, vocab=512, max_tokens=4096, max_batch=1024):
        g = torch.Generator().manual_seed(1)
        dt = cfg.torch_dtype
        randn = lambda *s: (torch.randn(s, generator=g) / math.sqrt(s[0])).to(dt)  # noqa: E731
        self.cfg, self.q_heads, self.kv_heads, self.head_dim = cfg, q_heads, kv_heads, head_dim
        self.embed = torch.randn((vocab, cfg.d), generator=g).to(dt).to(DEV)
        self.table = attn.rope_table(max_tokens, head_dim, scaling="linear", factor=2.0, device=DEV)
        self.width = (q_heads + 2 * kv_heads) * head_dim
        self.blocks = []
        for i in range(layers):
            qkv, out = randn(cfg.d, self.width), randn(q_heads * head_dim, cfg.d)
            pack = lambda w: moe.pack_weights(w[None].to(DEV), None, 16, 0)  # noqa: E731
            experts = moe.Layer(moe.PackedLayer.from_weights(cfg, synth.layer_weights(cfg, i), DEV), max_batch)
            self.blocks.append((pack(qkv), pack(out), experts))

    def norm(self, x):
        y = x.float()
        return (y * torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-6)).to(x.dtype)

    def linear(self, x, w, n):
        return moe.grouped_gemm(x, w, 16, 1, x.shape[1], n, 0, None, "none", x.dtype)

    def forward(self, tokens, cache, cu, seqs, start, pos, mask=None):
        """Final hidden states of the packed new tokens, and their routed experts (layers, tokens, k)."""
        x, routed = self.embed[tokens], []
        hq, hk, d = self.q_heads, self.kv_heads, self.head_dim
        for i, (w_qkv, w_out, experts) in enumerate(self.blocks):
            q, k, v = self.linear(self.norm(x), w_qkv, self.width).unflatten(1, (-1, d)).split([hq, hk, hk], 1)
            q = cache.append(k, v, cu, seqs, start, layer=i, q=q, pos=pos, cos_sin=self.table)
            y = attn.attention(q, cache, cu, seqs, start, mask=mask, layer=i)
            x = x + self.linear(y.flatten(1), w_out, self.cfg.d)
            x = x + experts.forward(self.norm(x))
            routed.append(experts.routing(x.shape[0])["ids"].clone())
        return self.norm(x), torch.stack(routed)

    def logits(self, hidden):
        return hidden.float() @ self.embed.float().T


def draft_tree(ranked, width=3, depth=3):
    """A tree over the model's ranking of the last token: `width` first guesses, each continued by the best ones.
    Returns (tokens, parents); parents index the drafted tokens, the root is the last verified token (index 0)."""
    tokens, parents = [], []
    for w in range(width):
        parent = 0
        for d in range(depth):
            tokens.append(ranked[w if d == 0 else (w + d) % len(ranked)])
            parents.append(parent)
            parent = len(tokens)
    return tokens, parents


def generate(prompts, rounds=4, layers=2):
    """Returns (model, cache, generated tokens per sequence, tokens accepted per round, expert counts)."""
    cfg = synth.CONFIGS["tiny"]
    m = Decoder(cfg, layers)
    n = len(prompts)
    cache = attn.KVCache.create(layers, pages=256, page_size=16, kv_heads=m.kv_heads, head_dim=m.head_dim, slots=n, max_pages=64,
                                dtype=cfg.torch_dtype, device=DEV)
    seqs = ints(list(range(n)))
    cu_list = [sum(map(len, prompts[:i])) for i in range(n + 1)]
    start = cache.extend(seqs, ints([len(p) for p in prompts]))
    pos = torch.cat([torch.arange(len(p), dtype=torch.int32) for p in prompts]).to(DEV)
    hidden, _ = m.forward(torch.tensor(sum(prompts, []), device=DEV), cache, ints(cu_list), seqs, start, pos)
    ranked = m.logits(hidden[[c - 1 for c in cu_list[1:]]]).topk(8).indices.tolist()
    last = [r[0] for r in ranked]                    # verified by the model, not yet in the cache
    out, accepted = [[t] for t in last], []
    counts = torch.zeros((layers, cfg.E), dtype=torch.int32, device=DEV)

    for _ in range(rounds):
        # every sequence's rows: the last verified token, then its tree
        toks, parents, cu = [], [], [0]
        trees = []
        for b in range(n):
            t, p = draft_tree(ranked[b])
            trees.append((t, p))
            toks += [last[b]] + t
            parents += [-1] + p
            cu.append(len(toks))
        size = [c1 - c0 for c0, c1 in zip(cu, cu[1:])]
        start = cache.extend(seqs, ints(size))
        mask, pos = attn.tree_mask(ints(parents), ints(cu), start, max(size))
        hidden, routed = m.forward(torch.tensor(toks, device=DEV), cache, ints(cu), seqs, start, pos, mask)
        moe.elb_accumulate(routed.contiguous(), cfg.E, counts)
        ranking = m.logits(hidden).topk(8).indices.tolist()
        keeps = []
        for b, (t, p) in enumerate(trees):
            at, keep = 0, [0]                        # follow the model's own choice down the tree
            while True:
                want = ranking[cu[b] + at][0]
                nxt = [i + 1 for i in range(len(t)) if p[i] == at and t[i] == want]
                if not nxt:
                    break
                at = nxt[0]
                keep.append(at)
                out[b].append(want)
            ranked[b] = ranking[cu[b] + at]
            last[b] = ranked[b][0]
            out[b].append(last[b])
            keeps.append(keep)
        accepted.append([len(k) for k in keeps])
        cache.compact(seqs, start, ints([sum(map(len, keeps[:i])) for i in range(n + 1)]), ints(sum(keeps, [])))
    return m, cache, out, accepted, counts


def main():
    rounds = int(sys.argv[1]) if len(sys.argv) > 1 else 4
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, 512, (k,), generator=g).tolist() for k in (5, 40, 17)]
    _, cache, out, accepted, counts = generate(prompts, rounds)
    for b, toks in enumerate(out):
        print(f"sequence {b}: {len(prompts[b])} prompt tokens, {len(toks)} generated: {toks}")
    print("tokens kept per round:", accepted)
    print("tokens in the cache:", cache.lens.tolist(), "pages held:", int((cache.refs > 0).sum()))
    print("most used experts:", [t.tolist() for t in moe.elb_topm(counts, 3)[0]])


if __name__ == "__main__":
    main()
