"""Float64 oracle of the attention half: rotary positions, the paged cache's bookkeeping, attention.

Plain CPU code written from the definitions in include/moe.h, one row or page at a time."""
from __future__ import annotations

import math

import torch


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0):
    """(frequencies, factor of cosines and sines)."""
    scale = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            g = min(max((original * f / (2 * math.pi) - 1.0) / 31.0, 0.0), 1.0)
            f *= g + (1.0 - g) / factor
            scale = 0.1 * math.log(factor) + 1.0
        out.append(f)
    return out, scale


def rope_table(positions, rot, **kw):
    f, scale = rope_frequencies(rot, **kw)
    return torch.tensor([[scale * math.cos(p * x) for x in f] + [scale * math.sin(p * x) for x in f] for p in positions],
                        dtype=torch.float64)


def rope(x, pos, table, interleaved=False, inverse=False):
    """x (T, H, D) -> float64; rows whose position the table lacks get NaN in the rotated part."""
    y = x.double().clone()
    rot = table.shape[1]
    for t, p in enumerate(pos.tolist()):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            inside = 0 <= p < table.shape[0]
            c = float(table[p, i]) if inside else math.nan
            s = float(table[p, rot // 2 + i]) if inside else math.nan
            s = -s if inverse else s
            xa, xb = x[t, :, a].double(), x[t, :, b].double()
            y[t, :, a], y[t, :, b] = xa * c - xb * s, xa * s + xb * c
    return y


class Cache:
    """The cache's bookkeeping on Python lists; page contents are (layers, 2, kv_heads, page_size, head_dim) tensors."""

    def __init__(self, pool, slots, max_pages):
        self.pool = pool.clone()             # (layers, pages, 2, H, ps, D)
        self.ps, self.max_pages = pool.shape[4], max_pages
        self.table = [[] for _ in range(slots)]
        self.lens = [0] * slots
        self.refs = [0] * pool.shape[1]

    def pages_for(self, n):
        return -(-n // self.ps)

    def extend(self, seqs, new):
        ok = [0 <= q < len(self.lens) and m >= 0 for q, m in zip(seqs, new)]
        plan, taken = [], 0
        free = [p for p, r in enumerate(self.refs) if r == 0]
        for q, m, good in zip(seqs, new, ok):
            if not good:
                plan.append(None)
                continue
            n = self.lens[q]
            shared = m > 0 and n % self.ps != 0 and self.refs[self.table[q][-1]] > 1
            need = self.pages_for(n + m) - self.pages_for(n) + shared
            if self.pages_for(n + m) > self.max_pages or taken + need > len(free):
                return [-1] * len(seqs)
            plan.append((shared, free[taken:taken + need]))
            taken += need
        start, dropped = [], []
        for q, m, p in zip(seqs, new, plan):
            if p is None:
                start.append(-1)
                continue
            shared, pages = p
            if shared:
                old = self.table[q].pop()
                self.pool[:, pages[0]] = self.pool[:, old]
                dropped.append(old)
            self.table[q] += pages
            for x in pages:
                self.refs[x] = 1
            start.append(self.lens[q])
            self.lens[q] += m
        for x in dropped:
            self.refs[x] -= 1
        return start

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            if not (0 <= s < len(self.lens) and 0 <= d < len(self.lens)) or s == d or self.lens[d]:
                continue
            self.table[d], self.lens[d] = list(self.table[s]), self.lens[s]
            for p in self.table[s]:
                self.refs[p] += 1

    def _cut(self, q, n):
        while len(self.table[q]) > self.pages_for(n):
            self.refs[self.table[q].pop()] -= 1
        self.lens[q] = n

    def free(self, seqs):
        for q in seqs:
            if 0 <= q < len(self.lens):
                self._cut(q, 0)

    def at(self, q, pos):
        return self.table[q][pos // self.ps], pos % self.ps

    def compact(self, seqs, start, keeps):
        for q, s, keep in zip(seqs, start, keeps):
            if not 0 <= q < len(self.lens) or s < 0 or s + len(keep) > self.lens[q]:
                continue
            for j, i in enumerate(keep):
                p, x = self.at(q, s + i)
                p2, x2 = self.at(q, s + j)
                self.pool[:, p2, :, :, x2] = self.pool[:, p, :, :, x].clone()
            self._cut(q, s + len(keep))

    def append(self, k, v, cu, seqs, start):
        """k, v (layers, T, H, D) already rotated."""
        for b, (q, s) in enumerate(zip(seqs, start)):
            if s < 0:
                continue
            for r in range(cu[b], cu[b + 1]):
                p, x = self.at(q, s + r - cu[b])
                self.pool[:, p, 0, :, x] = k[:, r]
                self.pool[:, p, 1, :, x] = v[:, r]

    def table_tensor(self):
        return torch.tensor([t + [-1] * (self.max_pages - len(t)) for t in self.table], dtype=torch.int32)


def tree_mask(parents, cu, start, words):
    """([set of visible drafted tokens] per row, positions)."""
    see, pos = [], []
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        rows = []
        for i in range(n):
            p = parents[cu[b] + i]
            good = -1 <= p < i and i < 32 * words and (p < 0 or bool(rows[p]))
            rows.append((rows[p] if p >= 0 else set()) | {i} if good else set())
        see += rows
        pos += [start[b] + max(len(x) - 1, 0) for x in rows]
    return see, pos


def bits(see, words):
    out = []
    for s in see:
        row = [0] * words
        for j in s:
            row[j // 32] |= 1 << (j % 32)
        out.append([w - (1 << 32) if w >= 1 << 31 else w for w in row])
    return torch.tensor(out, dtype=torch.int32).reshape(len(see), words)


def attention(q, k, v, see, scale):
    """One sequence: q (m, Hq, D), k/v (Hk, n, D), see: visible key indices of each row.  Only visible keys are touched.
    Returns out, lse, and for error bounds sum_j p_j |v_j| and max_j scale sum_d |q_d k_jd|."""
    m, hq, d = q.shape
    grp = hq // k.shape[0]
    out = torch.zeros(m, hq, d, dtype=torch.float64)
    lse = torch.full((m, hq), -math.inf, dtype=torch.float64)
    mag = torch.zeros(m, hq, d, dtype=torch.float64)
    smax = torch.zeros(m, hq, dtype=torch.float64)
    kd, vd, qd = k.double(), v.double(), q.double()
    for i in range(m):
        idx = torch.as_tensor(see[i], dtype=torch.long)
        if idx.numel() == 0:
            continue
        ki, vi = kd[:, idx], vd[:, idx]                                   # Hk, n, D
        x = qd[i].reshape(-1, grp, d)                                     # Hk, G, D
        s = torch.einsum("hgd,hnd->hgn", x, ki) * scale
        lse[i] = s.logsumexp(2).reshape(-1)
        p = s.softmax(2)
        out[i] = torch.einsum("hgn,hnd->hgd", p, vi).reshape(hq, d)
        mag[i] = torch.einsum("hgn,hnd->hgd", p, vi.abs()).reshape(hq, d)
        smax[i] = (torch.einsum("hgd,hnd->hgn", x.abs(), ki.abs()) * scale).amax(2).reshape(-1)
    return out, lse, mag, smax
