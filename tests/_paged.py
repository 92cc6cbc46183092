"""A paged cache's bookkeeping as a plain model on lists, and problems for the paged tests."""
from __future__ import annotations

import torch


class Book:
    """Page table, reference counts and lengths; one method per page operation."""

    def __init__(self, B, max_pages, n_pages, page_size):
        self.table = [[-1] * max_pages for _ in range(B)]
        self.ref = [0] * n_pages
        self.lens = [0] * B
        self.ps = page_size

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            if a < 0:
                continue
            self.table[b] = list(self.table[a])
            self.lens[b] = self.lens[a]
            for p in self.table[b]:
                if p >= 0:
                    self.ref[p] += 1

    def reserve(self, n_new):
        """(copy_src, copy_dst), or None if the pages do not suffice (nothing changes then)."""
        ps, B = self.ps, len(self.lens)
        table, ref, lens = [list(r) for r in self.table], list(self.ref), list(self.lens)
        src, dst = [-1] * B, [-1] * B
        for b in range(B):
            n, add = lens[b], n_new[b]
            if add <= 0:
                continue
            if n + add > len(table[b]) * ps:
                return None
            if n % ps and ref[table[b][n // ps]] > 1:
                if 0 not in ref:
                    return None
                src[b], dst[b] = table[b][n // ps], ref.index(0)
                ref[src[b]] -= 1
                ref[dst[b]] = 1
                table[b][n // ps] = dst[b]
            for t in range(-(-n // ps), -(-(n + add) // ps)):
                if 0 not in ref:
                    return None
                table[b][t] = ref.index(0)
                ref[table[b][t]] = 1
            lens[b] = n + add
        self.table, self.ref, self.lens = table, ref, lens
        return src, dst

    def release(self, ended, window, sinks):
        ps = self.ps
        for b, row in enumerate(self.table):
            for t, p in enumerate(row):
                behind = window > 0 and t * ps >= sinks and (t + 1) * ps <= self.lens[b] - window
                if p >= 0 and (ended[b] or behind):
                    self.ref[p] -= 1
                    row[t] = -1
            if ended[b]:
                self.lens[b] = 0

    def compact(self, max_moves):
        live = [p for p, r in enumerate(self.ref) if r > 0]
        holes = [p for p in range(len(live)) if self.ref[p] == 0]
        moves = [p for p in live if p >= len(live)]
        src, dst = moves[:max_moves], holes[:max_moves]
        to = dict(zip(src, dst))
        for p, h in to.items():
            self.ref[h], self.ref[p] = self.ref[p], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return src, dst


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(n_pages, Hkv, page, d, nhd, fill=float("nan")):
    """A K or V pool [n_pages, Hkv, page, d]; nhd: the heads inside a page's rows."""
    if nhd:
        return torch.full((n_pages, page, Hkv, d), fill, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    return torch.full((n_pages, Hkv, page, d), fill, dtype=torch.bfloat16, device="cuda")


def seen_mask(pos, t, window, sinks):
    """[queries, tokens]: whether the query at pos sees token t."""
    m = t[None, :] <= pos[:, None]
    if window:
        m &= (t[None, :] > pos[:, None] - window) | (t[None, :] < sinks)
    return m


def attention64(Q, K, V, pos, t, window, sinks, scale):
    """(o, sum p|v| / sum p, lse) in 64 bits of Q [n, Hq, d] over K, V [Hkv, T, d] at tokens t."""
    n, Hq, d = Q.shape
    Hkv = K.shape[0]
    q = Q.double().view(n, Hkv, Hq // Hkv, d)
    m = seen_mask(pos, t, window, sinks)[:, None, None, :]
    z = torch.einsum("nhgd,htd->nhgt", q, K.double()) * scale
    z = z.masked_fill(~m, -torch.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.where(m, torch.exp(z - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    o = torch.einsum("nhgt,htd->nhgd", p, V.double())
    a = torch.einsum("nhgt,htd->nhgd", p, V.double().abs())
    return o.reshape(n, Hq, d), a.reshape(n, Hq, d), lse.reshape(n, Hq)
