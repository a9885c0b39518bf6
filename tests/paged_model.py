"""A plain model of the paged pool: sequences one at a time, pages in Python lists, and
attention from the formula in 64 bits.  Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch


def ceil_div(a, b):
    return -(-a // b)


class PoolModel:
    """Tables, holders, lengths and page contents after each operation; `err` is the set of
    error codes the operation may have recorded first (empty: none)."""

    def __init__(self, n_pages, page, max_seqs, max_len, slab: torch.Tensor):
        self.n_pages, self.page, self.max_seqs, self.max_len = n_pages, page, max_seqs, max_len
        self.cols = ceil_div(max_len, page)
        self.len = [0] * max_seqs
        self.tab = [[] for _ in range(max_seqs)]
        self.slab = slab.clone()
        self.err = set()

    # -- views
    def table(self):
        return torch.tensor([t + [-1] * (self.cols - len(t)) for t in self.tab], dtype=torch.int32).view(
            self.max_seqs, self.cols)

    def refs(self):
        r = [0] * self.n_pages
        for t in self.tab:
            for x in t:
                r[x] += 1
        return r

    def free_pages(self):
        return [i for i, r in enumerate(self.refs()) if r == 0]

    def _listed(self, seqs):
        """(entry, sequence) of the entries to process; bad and repeated ones are recorded."""
        seen, out = set(), []
        for i, s in enumerate(seqs):
            if s == -1:
                continue
            if not 0 <= s < self.max_seqs or s in seen:
                self.err.add(-1)
                continue
            seen.add(s)
            out.append((i, s))
        return out

    # -- operations
    def reserve(self, seqs, grow):
        self.err = set()
        todo = []
        for i, s in self._listed(seqs):
            if grow[i] < 0:
                self.err.add(-1)
            elif self.len[s] + grow[i] > self.max_len:
                self.err.add(-5)
            elif grow[i] > 0:
                todo.append((s, grow[i]))
        tab, refs, free = [list(t) for t in self.tab], self.refs(), self.free_pages()
        copies = []
        for s, g in todo:
            ln = self.len[s]
            for c in range(ln // self.page, ceil_div(ln + g, self.page)):
                old = tab[s][c] if c < len(tab[s]) else -1
                if old >= 0 and refs[old] == 1:
                    continue
                if not free:
                    self.err.add(-5)
                    return
                x = free.pop(0)
                refs[x] = 1
                if old < 0:
                    assert len(tab[s]) == c
                    tab[s].append(x)
                else:
                    refs[old] -= 1
                    tab[s][c] = x
                    if c == ln // self.page:
                        copies.append((old, x, ln % self.page))
        self.tab = tab
        for old, x, rows in copies:
            self.slab[x, :, :, :, :rows] = self.slab[old, :, :, :, :rows]

    def fork(self, src, dst, deep=False):
        self.err = set()
        seen, todo = set(), []
        for a, b in zip(src, dst):
            if b == -1:
                continue
            if not 0 <= b < self.max_seqs or b in seen:
                self.err.add(-1)
                continue
            seen.add(b)
            if a == -1:
                continue
            if not 0 <= a < self.max_seqs or b in src:
                self.err.add(-1)
            elif self.len[b] or self.tab[b]:
                self.err.add(-6)
            else:
                todo.append((a, b))
        if deep:
            free = self.free_pages()
            if sum(ceil_div(self.len[a], self.page) for a, _ in todo) > len(free):
                self.err.add(-5)
                return
        for a, b in todo:
            held = self.tab[a][:ceil_div(self.len[a], self.page)]
            self.len[b] = self.len[a]
            if deep:
                own = [free.pop(0) for _ in held]
                for x, y in zip(held, own):
                    self.slab[y] = self.slab[x]
                self.tab[b] = own
            else:
                self.tab[b] = held

    def free(self, seqs, keep=None):
        self.err = set()
        for i, s in self._listed(seqs):
            k = 0 if keep is None else keep[i]
            if not 0 <= k <= self.len[s]:
                self.err.add(-1)
                continue
            self.tab[s] = self.tab[s][:ceil_div(k, self.page)]
            self.len[s] = k

    def compact(self):
        self.err = set()
        refs = self.refs()
        used = sum(r > 0 for r in refs)
        holes = [i for i in range(used) if refs[i] == 0]
        moved = [i for i in range(used, self.n_pages) if refs[i] > 0]
        to = dict(zip(moved, holes))
        for a, b in to.items():
            self.slab[b] = self.slab[a]
        self.tab = [[to.get(x, x) for x in t] for t in self.tab]
        return used

    def _writable(self, s, lo, hi):
        refs = self.refs()
        if hi > self.max_len:
            return -5
        held = [self.tab[s][c] if c < len(self.tab[s]) else -1 for c in range(lo // self.page, ceil_div(hi, self.page))]
        if any(x < 0 for x in held):
            return -5
        return -6 if any(refs[x] > 1 for x in held) else 0

    def write(self, layer, k, v, seqs, start, count, total, most):
        self.err = set()
        for i, s in enumerate(seqs):
            if s == -1 or count[i] == 0:
                continue
            if not 0 <= s < self.max_seqs or s in seqs[:i]:
                self.err.add(-1)
                continue
            if count[i] < 0 or count[i] > most or start[i] < 0 or start[i] + count[i] > total:
                self.err.add(-1)
                continue
            e = self._writable(s, self.len[s], self.len[s] + count[i])
            if e:
                self.err.add(e)
                continue
            for r in range(count[i]):
                p = self.len[s] + r
                x = self.tab[s][p // self.page]
                self.slab[x, layer, 0, :, p % self.page] = k[start[i] + r]
                self.slab[x, layer, 1, :, p % self.page] = v[start[i] + r]

    def advance(self, seqs, count):
        self.err = set()
        for i, s in self._listed(seqs):
            if count[i] < 0:
                self.err.add(-1)
            elif count[i]:
                to = self.len[s] + count[i]
                if to > self.max_len or len(self.tab[s]) < ceil_div(to, self.page):
                    self.err.add(-5)
                else:
                    self.len[s] = to

    def rows_of(self, s, n):
        """[L, 2, nkv, n, d] of positions [0, n)."""
        pages = self.slab[torch.tensor(self.tab[s][:ceil_div(n, self.page)], dtype=torch.long, device=self.slab.device)]
        return pages.permute(1, 2, 3, 0, 4, 5).flatten(3, 4)[:, :, :, :n] if n else \
            self.slab[:0].permute(1, 2, 3, 0, 4, 5).flatten(3, 4)


def attention(q, k, v, pos, causal, window, sinks):
    """Rows q [R, nq, d] at positions pos over keys k, v [nkv, n, d], in 64 bits: the outputs and, per
    element, the weighted mean of |v| and the largest error of a score in fp32 (for error bounds)."""
    q, k, v = q.double(), k.double(), v.double()
    R, nq, d = q.shape
    nkv, n, _ = k.shape
    j = torch.arange(n, device=q.device)[None]
    i = torch.tensor(pos, device=q.device)[:, None]
    see = torch.ones(R, n, dtype=torch.bool, device=q.device)
    if causal:
        see &= j <= i
    if window:
        see &= (j < sinks) | (j > i - window)
    out, mean, score = torch.empty_like(q), torch.empty_like(q), torch.empty(R, nq, 1, dtype=q.dtype, device=q.device)
    for h in range(nq):
        g = h // (nq // nkv)
        # unseen keys and values may hold anything
        t = torch.where(see, q[:, h] @ torch.where(see.any(0)[:, None], k[g], 0).T / math.sqrt(d), -math.inf)
        w = torch.softmax(t, 1)
        vv = torch.where(see.any(0)[:, None], v[g], 0)
        out[:, h] = w @ vv
        mean[:, h] = w @ vv.abs()
        kk = torch.where(see.any(0)[:, None], k[g].abs(), 0)
        score[:, h, 0] = (q[:, h].abs() @ kk.T / math.sqrt(d)).amax(1)
    return out, mean, score


def bound(out, mean, score, n, d, dtype):
    """Largest distance of a kernel's output from the formula's, per element.

    Scores: d products and sums in fp32, each off by at most 2^-23 (a tensor core may
    truncate) of sum |q k| / sqrt(d), so a weight is off by a factor of at most
    1 + 2 d 2^-23 score (e^x - 1 <= 2x for x <= 1), the same for numerator and
    denominator: twice that.  2^x: 2^-21.  Sums over n keys: n 2^-23 each.  bf16: each
    weight is rounded (2^-8), and so is the result (2^-8 of it); fp32: the result 2^-24."""
    f32 = 2 * (2 * d * 2.0 ** -23 * score) + 2.0 ** -20 + 2 * n * 2.0 ** -23
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    p = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    e = (p + f32) * mean
    return e + half * (out.abs() + e) + 1e-30


def np_i32(t):
    return t.cpu().numpy().astype(np.int64)
