"""Sequences that gave tokens back: seq_lens lowered between two page calls (speculated tokens that were rejected,
a sequence begun anew).  The pages past the shorter length are the sequence's own until they are exchanged."""
from __future__ import annotations

import random
from collections import Counter

import pytest
import torch

import token_level_sparse_jssa_b200 as jssa
from tests._paged import Book, i32

pytestmark = pytest.mark.gpu


class Rollback(Book):
    """The model with entries past a sequence's length: what reserve and fork write over is given up first."""

    def reserve(self, n_new):
        kept = [list(r) for r in self.table], list(self.ref)
        for b, add in enumerate(n_new):
            lo, hi = -(-self.lens[b] // self.ps), -(-(self.lens[b] + add) // self.ps)
            for t in range(lo, hi) if add > 0 and hi <= len(self.table[b]) else ():
                if self.table[b][t] >= 0:
                    self.ref[self.table[b][t]] -= 1
                    self.table[b][t] = -1
        got = super().reserve(n_new)
        if got is None:
            self.table, self.ref = kept
        return got

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            if a < 0:
                continue
            used = -(-self.lens[a] // self.ps)
            for p in self.table[b]:
                if p >= 0:
                    self.ref[p] -= 1
            self.table[b] = self.table[a][:used] + [-1] * (len(self.table[a]) - used)
            self.lens[b] = self.lens[a]
            for p in self.table[b]:
                if p >= 0:
                    self.ref[p] += 1


def _start(book):
    table, ref, lens = i32(book.table), i32(book.ref), i32(book.lens)
    K = torch.zeros(len(book.ref), 1, book.ps, 64, dtype=torch.bfloat16, device="cuda")
    L = jssa.make_paged_layout(K, K, table, 1)
    return table, ref, lens, L, jssa.alloc_paged_workspace(L)


def _same(book, table, ref, lens):
    torch.cuda.synchronize()
    assert table.tolist() == book.table and ref.tolist() == book.ref and lens.tolist() == book.lens


def test_a_full_pool_serves_a_sequence_that_gave_tokens_back():
    # 2 sequences hold all 6 pages; one gives 30 tokens back and takes them again, for ever
    book = Rollback(2, 3, 6, 16)
    book.reserve([48, 48])
    table, ref, lens, L, ws = _start(book)
    src, dst = i32([0, 0]), i32([0, 0])
    for _ in range(4):
        book.lens[0] = 18
        lens[0] = 18
        jssa.pages_reserve(L, i32([30, 0]), table, ref, lens, src, dst, ws)
        assert jssa.read_device_status(ws) == (0, 0)
        assert book.reserve([30, 0]) == ([-1, -1], [-1, -1])
        _same(book, table, ref, lens)
    assert ref.tolist() == [1] * 6


def test_a_refused_reserve_changes_nothing_after_a_rollback():
    book = Rollback(2, 4, 6, 16)
    book.reserve([48, 48])
    table, ref, lens, L, ws = _start(book)
    book.lens[0] = lens[0] = 18
    src, dst = i32([0, 0]), i32([0, 0])
    jssa.pages_reserve(L, i32([40, 16]), table, ref, lens, src, dst, ws)   # 3 pages, of which 1 is its own
    assert jssa.read_device_status(ws) == (5, jssa.DEV_NO_PAGES)
    _same(book, table, ref, lens)


@pytest.mark.parametrize("seed,B,mp,n_pages,ps", [(1, 5, 6, 24, 16), (2, 40, 9, 170, 32), (3, 300, 4, 900, 16),
                                                  (4, 1024, 3, 2500, 16), (5, 9, 300, 1500, 16)])
def test_page_operations_follow_the_model(seed, B, mp, n_pages, ps):
    r = random.Random(seed)
    book = Rollback(B, mp, n_pages, ps)
    table, ref, lens, L, ws = _start(book)
    src, dst = i32([0] * B), i32([0] * B)
    for step in range(40):
        op = r.choice(("grow", "grow", "back", "back", "fork", "release", "window"))
        if op == "grow":
            n_new = [r.choice((0, 0, 1, 1, 3, ps, r.randint(0, 3 * ps), r.randint(0, mp * ps // 2))) for _ in range(B)]
            n_new = [min(x, mp * ps - n) for x, n in zip(n_new, book.lens)]
            got = book.reserve(n_new)
            jssa.pages_reserve(L, i32(n_new), table, ref, lens, src, dst, ws)
            if got is None:
                assert jssa.read_device_status(ws) == (5, jssa.DEV_NO_PAGES)
                got = [-1] * B, [-1] * B
            assert (src.tolist(), dst.tolist()) == tuple(map(list, got))
        elif op == "back":
            book.lens = [max(0, n - r.choice((0, 1, 5, ps, 2 * ps, n))) if r.random() < 0.7 else n for n in book.lens]
            # a length ends in a page that is still there (pages behind a window are not)
            book.lens = [0 if n and row[(n - 1) // ps] < 0 else n for n, row in zip(book.lens, book.table)]
            lens.copy_(i32(book.lens))
        elif op == "fork":
            empty = [b for b in range(B) if book.lens[b] == 0]
            held = [b for b in range(B) if book.lens[b] > 0]
            if not empty or not held:
                continue
            r.shuffle(empty)
            b = empty[:r.randint(1, len(empty))]
            a = [r.choice(held + [-1]) for _ in b]
            book.fork(a, b)
            jssa.pages_fork(L, i32(a), i32(b), table, ref, lens, ws)
        else:
            ended = [int(op == "release" and r.random() < 0.4) for _ in range(B)]
            window, sinks = (0, 0) if op == "release" else (r.choice((20, ps)), r.choice((0, 4, ps + 1)))
            book.release(ended, window, sinks)
            jssa.pages_release(L, i32(ended), window, sinks, table, ref, lens, ws)
        _same(book, table, ref, lens)
        assert jssa.read_device_status(ws)[1] == 0, (step, op)
        named = Counter(p for row in book.table for p in row)
        assert book.ref == [named[p] for p in range(n_pages)]   # no page is lost, none counted twice
    jssa.pages_release(L, i32([1] * B), 0, 0, table, ref, lens, ws)
    torch.cuda.synchronize()
    assert not ref.any() and bool((table == -1).all())
