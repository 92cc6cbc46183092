"""The paged caches on the GPU: attention of the newest tokens against the formula in 64 bits,
the page operations against a model on lists, appends bit for bit, and all of them together."""
from __future__ import annotations

import random

import pytest
import torch

import token_level_sparse_jssa_b200 as jssa
from tests._paged import Book, attention64, i32, pool, seen_mask

pytestmark = pytest.mark.gpu

# Bound of an attention output, from the roundings it is made of.  With A = sum p|v| / sum p:
#   logits: products of bf16 are exact in fp32; a sum of d terms is off by at most d 2^-24 times
#     the sum of their magnitudes.  With the inputs below that is under 256 2^-24 * 46 < 2^-10
#     in the logit (|q||k| sm_scale <= 46 at d = 256), and the softmax's subtraction, product
#     and exponential add less than 2^-17.  A relative error of 2^-10 of every p moves sum p v
#     by at most 2^-10 A and sum p by 2^-10 of itself: 2^-9 A together.
#   p is rounded to bf16 before the product with v (by at most 2^-8 of p): 2^-8 A.
#   bf16 output: 2^-8 |o|.  fp32 sums over at most 2^14 visible tokens, in partial sums of at
#     most 2^11 terms that are merged: under 2^-10 A.
P_TOL = 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -10
OUT_TOL = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
LSE_TOL = 2.0 ** -9     # 2^-10 of the logits, 2^-10 of the fp32 sum


class Problem:
    """Sequences of lens[b] tokens, the last nq[b] of them new, over pools in which only rows
    that some new token sees are finite."""

    def __init__(self, lens, nq, d=128, Hkv=2, G=4, page=16, window=0, sinks=0, nhd=False, out=torch.bfloat16, seed=1,
                 fused=False, tail=0, extra_cols=1):
        self.lens, self.nq, self.d, self.Hkv, self.Hq, self.page = lens, nq, d, Hkv, Hkv * G, page
        self.window, self.sinks, self.out = window, sinks, out
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = random.Random(seed)
        B, mp = len(lens), max(1, -(-max(lens) // page)) + extra_cols
        need = [(b, t) for b in range(B) for t in range(-(-lens[b] // page))]
        self.n_pages = len(need) + 3
        ids = list(range(self.n_pages))
        r.shuffle(ids)
        self.K, self.V = pool(self.n_pages, Hkv, page, d, nhd), pool(self.n_pages, Hkv, page, d, nhd)
        table = [[-1] * mp for _ in range(B)]
        self.k64, self.v64, self.t, self.pos = [], [], [], []
        for b in range(B):
            pos = torch.arange(lens[b] - nq[b], lens[b], device="cuda")
            t = torch.arange(lens[b], device="cuda")
            t = t[seen_mask(pos, t, window, sinks).any(0)] if nq[b] else t[:0]
            k = torch.randn(len(t), Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
            k *= torch.where(torch.rand(len(t), 1, 1, generator=g, device="cuda") < 0.02, 2.0, 1.0).to(torch.bfloat16)
            v = torch.randn(len(t), Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
            rows = set((t // page).tolist())
            for (bb, s), p in zip(need, ids):
                if bb == b and s in rows:   # pages that no query sees stay out of the table
                    table[b][s] = p
            if len(t):
                at = torch.tensor(table[b], device="cuda")[t // page]
                self.K[at, :, t % page] = k
                self.V[at, :, t % page] = v
            self.k64.append(k.transpose(0, 1))
            self.v64.append(v.transpose(0, 1))
            self.t.append(t)
            self.pos.append(pos)
        self.table, self.seq_lens = i32(table), i32(lens)
        self.begin = [0]
        for x in nq:
            self.begin.append(self.begin[-1] + x)
        self.q_begin = i32(self.begin)
        self.n = self.begin[-1] + tail
        q = torch.randn(self.n, self.Hq + (5 if fused else 0), d, generator=g, device="cuda").to(torch.bfloat16)
        self.Q = q[:, :self.Hq]
        self.max_q = max(nq)
        self.scale = d ** -0.5
        self.L = jssa.make_paged_layout(self.K, self.V, self.table, self.Hq,
                                        jssa.OUT_BF16 if out == torch.bfloat16 else jssa.OUT_F32)
        self.ws = jssa.alloc_paged_workspace(self.L, self.max_q)
        self.O = torch.full((self.n, self.Hq, d), -777.0, dtype=out, device="cuda")
        self.lse = torch.full((self.n, self.Hq), -777.0, device="cuda")

    def run(self, lse=True, stream=None):
        jssa.paged_attn(self.L, self.Q, self.K, self.V, self.table, self.q_begin, self.max_q, self.seq_lens,
                        self.window, self.sinks, self.scale, self.O, self.lse if lse else None, self.ws, stream)
        return self.O

    def check(self, flags=0, keep=None, skip=()):
        torch.cuda.synchronize()
        assert jssa.read_device_status(self.ws)[1] == flags
        for b in range(len(self.lens)):
            lo, hi = self.begin[b], self.begin[b + 1]
            o, lse = self.O[lo:hi], self.lse[lo:hi]
            if b in skip:
                assert bool((o == -777.0).all()) and bool((lse == -777.0).all())
                continue
            if lo == hi:
                continue
            k, v, t = self.k64[b], self.v64[b], self.t[b]
            if keep is not None:
                k, v, t = k[:, keep[b]], v[:, keep[b]], t[keep[b]]
            for i in range(0, hi - lo, 512):
                want, a, z = attention64(self.Q[lo:hi][i:i + 512], k, v, self.pos[b][i:i + 512], t, self.window,
                                         self.sinks, self.scale)
                got = o[i:i + 512].double()
                bad = (got - want).abs() > P_TOL * a + OUT_TOL[self.out] * want.abs()
                assert not bool(bad.any()) and bool(torch.isfinite(got).all()), \
                    (b, i, int(bad.sum()), float((got - want).abs().max()))
                gl = lse[i:i + 512].double()
                assert torch.equal(gl.isinf(), z.isinf())
                assert bool(((gl - z).abs() <= LSE_TOL)[~z.isinf()].all())
        tail = slice(self.begin[-1], self.n)
        assert bool((self.O[tail] == -777.0).all()) and bool((self.lse[tail] == -777.0).all())


CASES = [
    # single tokens
    dict(lens=[1], nq=[1]),
    dict(lens=[1, 2, 16, 17, 127, 128, 129, 300], nq=[1] * 8, page=16),
    dict(lens=[0, 5, 0, 1000], nq=[0, 1, 0, 1], page=32),
    dict(lens=[2048], nq=[1], d=64, Hkv=1, G=16, page=64),
    dict(lens=[700, 1500], nq=[1, 1], d=256, Hkv=3, G=2, page=64, window=1024, sinks=4),
    dict(lens=[5000, 37, 3000], nq=[1, 1, 1], Hkv=8, G=1, page=128),
    dict(lens=[4097], nq=[1], Hkv=1, G=128, page=256),
    dict(lens=[9000], nq=[1], d=64, Hkv=5, G=7, page=48),
    dict(lens=[16000], nq=[1], d=128, Hkv=1, G=1, page=4096),
    # few tokens
    dict(lens=[100, 9, 260, 33], nq=[3, 9, 1, 16], d=64, G=3, page=48, nhd=True),
    dict(lens=[2000, 2000], nq=[8, 5], window=100, sinks=0, fused=True),
    dict(lens=[2000, 40], nq=[8, 5], d=256, G=1, window=16, sinks=33, page=16),
    dict(lens=[600, 601, 602], nq=[2, 0, 4], G=8, Hkv=1, window=1, sinks=1, tail=3),
    dict(lens=[600, 700], nq=[2, 4], G=8, Hkv=1, window=1, sinks=0),
    dict(lens=[900, 18, 333], nq=[17, 17, 2], d=64, Hkv=2, G=1, window=100, sinks=20, page=48),
    dict(lens=[700, 16, 2000], nq=[16, 16, 9], d=64, G=2, page=32, fused=True),
    dict(lens=[1300, 31, 65], nq=[4, 1, 3], G=8, Hkv=1, window=70, sinks=3, page=16, tail=2),
    dict(lens=[1300, 31, 65], nq=[1, 1, 0], G=27, Hkv=2, page=80),
    dict(lens=[800, 20], nq=[16, 3], d=256, Hkv=2, G=1, window=40, sinks=17, page=16),
    # chunks and whole prompts
    dict(lens=[257], nq=[257], Hkv=1, G=1),
    dict(lens=[513, 64, 1], nq=[513, 64, 1], d=64, G=2, page=32),
    dict(lens=[1000, 300, 1200], nq=[400, 3, 130], G=4, page=64, fused=True, tail=9),
    dict(lens=[900, 450], nq=[500, 1], d=256, Hkv=1, G=2, page=128, nhd=True),
    dict(lens=[1500, 77], nq=[700, 77], d=64, Hkv=2, G=8, window=600, sinks=5, page=32, nhd=True),
    dict(lens=[1500, 700], nq=[300, 700], Hkv=1, G=12, window=130, sinks=100, page=16),
    dict(lens=[800], nq=[800], d=256, Hkv=2, G=1, window=64, sinks=70, page=16),
    dict(lens=[3000], nq=[129], Hkv=2, G=1, window=5000, sinks=4, page=112),
    dict(lens=[700], nq=[65], Hkv=1, G=128, page=16),
    dict(lens=[600] * 40, nq=[1 + 7 * (i % 9) for i in range(40)], d=64, Hkv=1, G=5, page=16),
]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", CASES)
def test_attention_matches_the_formula(kw, out):
    p = Problem(**kw, out=out)
    p.run()
    p.check()
    first = p.O.clone()
    p.run()   # the workspace is ready for the next call, and the order of the sums is fixed
    p.check()
    assert torch.equal(first, p.O)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_logits_and_masked_rows(d):
    # logits up to about 300 apart: the running maximum moves often, far keys vanish
    p = Problem([1, 900, 400], [1, 300, 400], d=d, G=2, page=16, window=200, sinks=3)
    order = torch.linspace(0.2, 3.0, p.n_pages, device="cuda")
    p.scale = 1.0
    p.K *= order.view(-1, 1, 1, 1).to(torch.bfloat16)
    for b in range(3):
        at = p.table[b].long()[p.t[b] // p.page]
        p.k64[b] = p.K[at, :, p.t[b] % p.page].transpose(0, 1)
    p.run()
    torch.cuda.synchronize()
    assert jssa.read_device_status(p.ws)[1] == 0
    for b in range(3):
        lo, hi = p.begin[b], p.begin[b + 1]
        want, a, z = attention64(p.Q[lo:hi], p.k64[b], p.v64[b], p.pos[b], p.t[b], p.window, p.sinks, 1.0)
        # the logits' own bound: d 2^-24 times the sum of the products' magnitudes
        mags = torch.einsum("nhgd,htd->nhgt", p.Q[lo:hi].double().abs().view(hi - lo, p.Hkv, -1, d),
                            p.k64[b].double().abs()).amax(-1).reshape(hi - lo, p.Hq, 1)
        tol = d * 2.0 ** -24 * mags + 2.0 ** -14
        err = (p.O[lo:hi].double() - want).abs()
        assert bool((err <= (P_TOL + 2 * tol.expm1()) * a + OUT_TOL[p.out] * want.abs()).all())
        assert bool(((p.lse[lo:hi].double() - z).abs()[..., None] <= tol + 2.0 ** -10 + z.abs()[..., None] * 2.0 ** -22)
                    .all())


def test_missing_pages_are_left_out_and_flagged():
    p = Problem([500, 300, 20], [40, 1, 20], page=16)
    keep = [torch.ones(len(t), dtype=torch.bool, device="cuda") for t in p.t]
    for b, s, page in ((0, 3, -1), (0, 30, p.n_pages), (1, 0, -5), (1, 18, 1 << 30), (2, 0, -1), (2, 1, -1)):
        p.table[b, s] = page
        keep[b] &= p.t[b] // p.page != s
    p.run()
    p.check(flags=jssa.DEV_BAD_INDEX, keep=keep)   # sequence 2 has nothing left: zeros and -inf
    assert bool((p.O[p.begin[2]:p.begin[3]] == 0).all())


def test_bad_sequences_are_left_out_and_flagged():
    for bad in (-1, 10 ** 6, 39):            # negative, past the table, fewer tokens than new ones
        p = Problem([500, 300, 260], [40, 40, 3], page=16)
        p.seq_lens[1] = bad
        p.run()
        p.check(flags=jssa.DEV_BAD_SEQ_LEN, skip=(1,))
    p = Problem([500, 300, 260], [40, 3, 30], page=16)
    p.max_q = 30                             # sequence 0 has more
    p.run()
    p.check(flags=jssa.DEV_BAD_SEQ_LEN, skip=(0,))
    p = Problem([500, 300, 260], [40, 3, 30], page=16)
    p.q_begin[3] = 10 ** 6                   # past the rows that are there
    p.run()
    p.check(flags=jssa.DEV_BAD_SEQ_LEN, skip=(2,))
    p = Problem([500, 300, 260], [40, 3, 30], page=16)
    p.q_begin[1] = 50                        # sequence 1 ends before it begins; sequence 0 takes rows past its own
    p.run(lse=False)
    torch.cuda.synchronize()
    assert jssa.read_device_status(p.ws)[1] == jssa.DEV_BAD_SEQ_LEN


def test_attention_without_lse_and_with_small_workspaces():
    p = Problem([500, 300], [140, 1])
    p.run(lse=False)
    torch.cuda.synchronize()
    assert bool((p.lse == -777.0).all())
    p.lse.fill_(0)
    p.run()
    p.check()
    with pytest.raises(jssa.JssaError) as e:
        jssa.paged_attn(p.L, p.Q, p.K, p.V, p.table, p.q_begin, p.max_q, p.seq_lens, 0, 0, p.scale, p.O, None,
                        p.ws[:256])
    assert e.value.code == 3


def test_binding_refuses_tensors_that_do_not_fit():
    p = Problem([50, 30], [4, 1])
    args = dict(Q=p.Q, K=p.K, V=p.V, page_table=p.table, q_begin=p.q_begin, max_q_len=4, seq_lens=p.seq_lens, window=0,
                n_sinks=0, sm_scale=0.1, O=p.O, lse=p.lse, ws=p.ws)
    for kw in (dict(Q=p.Q.float()), dict(Q=p.Q[:, :-1]), dict(Q=p.Q.transpose(0, 1)), dict(K=p.K[1:]), dict(V=p.V.float()),
               dict(K=pool(p.n_pages, p.Hkv, p.page, p.d, True)), dict(page_table=p.table.long()),
               dict(page_table=p.table[:, :-1]), dict(q_begin=p.q_begin[1:]), dict(seq_lens=p.seq_lens.cpu()),
               dict(O=p.O.float()), dict(O=p.O[:-1]), dict(lse=p.lse[:, 1:]), dict(lse=p.lse.half())):
        with pytest.raises(ValueError):
            jssa.paged_attn(p.L, **{**args, **kw})


@pytest.mark.parametrize("d", [64, 128, 256])
def test_pools_inside_one_tensor(d):
    # K and V of a page side by side in one tensor, rows with room behind them
    p = Problem([700, 45, 300], [130, 1, 5], d=d, Hkv=2, G=2, page=32)
    both = torch.full((p.n_pages, 2, 2, 32, d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    K, V = both[:, 0, :, :, :d], both[:, 1, :, :, 8:]
    assert V.data_ptr() % 16 == 0
    K.copy_(p.K)
    V.copy_(p.V)
    p.K, p.V = K, V
    p.L = jssa.make_paged_layout(K, V, p.table, p.Hq, jssa.OUT_BF16)
    p.run()
    p.check()
    new = torch.randn(136, 2, d, device="cuda").to(torch.bfloat16)
    jssa.paged_append_kv(p.L, new, new, K, V, p.table, p.q_begin, p.seq_lens, p.ws)
    for b in range(3):
        t = p.pos[b]
        at = p.table[b].long()[t // 32]
        assert torch.equal(K[at, :, t % 32], new[p.begin[b]:p.begin[b + 1]])
        assert torch.equal(V[at, :, t % 32], new[p.begin[b]:p.begin[b + 1]])
    assert bool(both[:, 0, :, :, d:].isnan().all()) and bool(both[:, 1, :, :, :8].isnan().all())


@pytest.mark.parametrize("kw", [
    dict(lens=[300], nq=[3], d=256, Hkv=1, G=128, page=48),
    dict(lens=[1000, 300], nq=[1, 2], d=64, Hkv=2, G=128, page=64, window=77, sinks=9),
    dict(lens=[16], nq=[16], d=64, Hkv=1, G=1, page=16, extra_cols=0),
    dict(lens=[500, 200], nq=[1, 200], window=2 ** 31 - 1, sinks=2 ** 31 - 1),
    dict(lens=[500, 200], nq=[1, 200], window=50, sinks=2 ** 31 - 1),
    dict(lens=[500, 200], nq=[1, 2], window=50, sinks=2 ** 31 - 1, G=2),
])
def test_extremes(kw):
    for out in (torch.bfloat16, torch.float32):
        p = Problem(**kw, out=out)
        p.run()
        p.check()


def test_bounds_on_new_tokens_may_be_generous():
    # max_q_len far above what the sequences bring: the large kernel for single tokens
    for lens, nq in (([700, 20, 5000], [1, 1, 1]), ([700, 20], [30, 2])):
        p = Problem(lens, nq, page=32)
        p.max_q = 100000
        p.ws = jssa.alloc_paged_workspace(p.L, p.max_q)
        p.run()
        p.check()


def test_rows_before_the_first_sequence_are_left():
    for nq in ([1, 2, 1], [40, 1, 130]):
        p = Problem([700, 20, 300], nq, tail=5)
        q, o, lse = p.Q, p.O, p.lse
        pad = torch.full_like(q[:3], float("nan"))
        p.Q = torch.cat([pad, q])
        p.O, p.lse = torch.cat([o[:3], o]), torch.cat([lse[:3], lse])
        p.q_begin += 3
        p.run()
        assert bool((p.O[:3] == -777.0).all()) and bool((p.lse[:3] == -777.0).all())
        p.Q, p.O, p.lse = q, p.O[3:], p.lse[3:]
        p.check()


def test_one_workspace_for_several_layouts():
    a, b = Problem([5000, 40], [1, 1], seed=4), Problem([900, 300, 8], [300, 1, 8], d=64, Hkv=1, G=2, page=48, seed=6)
    ws = max(a.ws, b.ws, key=len)
    a.ws = b.ws = ws
    K = torch.zeros(3000, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    book = Book(50, 20, 3000, 16)
    table, ref, lens = _state(book)
    L = jssa.make_paged_layout(K, K, table, 1)
    assert len(ws) >= jssa.paged_workspace_size(L)
    src, dst = i32([0] * 50), i32([0] * 50)
    r = random.Random(3)
    for step in range(6):
        n_new = [r.choice((0, 1, 7, 33)) for _ in range(50)]
        got = book.reserve(n_new)
        jssa.pages_reserve(L, i32(n_new), table, ref, lens, src, dst, ws)
        assert (src.tolist(), dst.tolist()) == got
        if step == 2:
            book.release([int(b % 3 == 0) for b in range(50)], 0, 0)
            jssa.pages_release(L, i32([int(b % 3 == 0) for b in range(50)]), 0, 0, table, ref, lens, ws)
            held = [b for b in range(50) if book.lens[b]]
            book.fork(held[:10], [0, 3, 6, 9, 12, 15, 18, 21, 24, 27])
            jssa.pages_fork(L, i32(held[:10]), i32([0, 3, 6, 9, 12, 15, 18, 21, 24, 27]), table, ref, lens, ws)
        for p in (a, b):
            p.O.fill_(-777.0)
            p.run()
            p.check()
        _same(book, table, ref, lens)


def test_many_pieces_and_many_sequences():
    # one item cut over the whole GPU; more sequences than the GPU has multiprocessors, most of one tile
    p = Problem([40000], [1], Hkv=1, G=2, page=64, out=torch.float32)
    p.run()
    p.check()
    r = random.Random(5)
    lens = [r.choice((1, 3, 60, 129, 400)) for _ in range(1024)]
    p = Problem(lens, [min(n, r.choice((0, 1, 1, 2))) for n in lens], d=64, Hkv=1, G=4, page=16)
    p.run()
    p.check()


# --------------------------------------------------------------------------- append
@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("d,Hkv,page", [(64, 1, 16), (128, 3, 48), (256, 2, 128)])
def test_append_writes_every_row_and_no_other(d, Hkv, page, nhd):
    lens, nq = [0, 1, page + 3, 5 * page, 400], [0, 1, 2, 5 * page, 77]
    B, mp = len(lens), 5 + 400 // page
    n_pages = B * mp
    K, V = pool(n_pages, Hkv, page, d, nhd, 3.0), pool(n_pages, Hkv, page, d, not nhd, 5.0)
    table = torch.randperm(n_pages, device="cuda").to(torch.int32).view(B, mp)
    begin = [0]
    for x in nq:
        begin.append(begin[-1] + x)
    new = torch.randn(begin[-1] + 4, 2 * Hkv + 1, d, device="cuda").to(torch.bfloat16)
    kn, vn = new[:, :Hkv], new[:, Hkv:2 * Hkv]
    L = jssa.make_paged_layout(K, V, table, Hkv)
    ws = jssa.alloc_paged_workspace(L)
    want_k, want_v = K.clone(), V.clone()
    for b in range(B):
        for i in range(nq[b]):
            t = lens[b] - nq[b] + i
            want_k[table[b, t // page], :, t % page] = kn[begin[b] + i]
            want_v[table[b, t // page], :, t % page] = vn[begin[b] + i]
    jssa.paged_append_kv(L, kn, vn, K, V, table, i32(begin), i32(lens), ws)
    assert jssa.read_device_status(ws)[1] == 0
    assert torch.equal(K, want_k) and torch.equal(V, want_v)


def test_append_leaves_out_bad_sequences_and_pages():
    K, V = pool(8, 2, 16, 64, False, 0.0), pool(8, 2, 16, 64, False, 0.0)
    table = i32([[0, 1], [2, -1], [3, 8], [4, 5]])
    rows = torch.ones(40, 2, 64, dtype=torch.bfloat16, device="cuda")
    L = jssa.make_paged_layout(K, V, table, 2)
    ws = jssa.alloc_paged_workspace(L)
    begin, lens = i32([0, 5, 15, 25, 35]), i32([33, 20, 20, 9])
    jssa.paged_append_kv(L, rows, rows, K, V, table, begin, lens, ws)
    assert jssa.read_device_status(ws)[1] == jssa.DEV_BAD_SEQ_LEN | jssa.DEV_BAD_INDEX
    assert K.sum((1, 3)).count_nonzero(1).tolist() == [0, 0, 6, 6, 0, 0, 0, 0]


# --------------------------------------------------------------------------- page operations
def _state(book):
    return i32(book.table), i32(book.ref), i32(book.lens)


def _same(book, table, ref, lens):
    torch.cuda.synchronize()
    assert table.tolist() == book.table and ref.tolist() == book.ref and lens.tolist() == book.lens


@pytest.mark.parametrize("seed,B,mp,n_pages,ps", [(1, 5, 6, 20, 16), (2, 40, 9, 150, 32), (3, 300, 4, 900, 16),
                                                  (4, 1024, 3, 2500, 16), (5, 64, 40, 33000, 16), (6, 1, 1, 1, 16),
                                                  (7, 1000, 70, 9000, 16)])
def test_page_operations_follow_the_model(seed, B, mp, n_pages, ps):
    r = random.Random(seed)
    book = Book(B, mp, n_pages, ps)
    table, ref, lens = _state(book)
    K = torch.zeros(n_pages, 1, ps, 64, dtype=torch.bfloat16, device="cuda")
    L = jssa.make_paged_layout(K, K, table, 1)
    ws = jssa.alloc_paged_workspace(L)
    src, dst, n_moves = i32([0] * B), i32([0] * B), i32([0])
    refused = 0
    for step in range(40):
        op = r.choice(("grow", "grow", "fork", "release", "window", "compact"))
        if op == "grow":
            n_new = [r.choice((0, 0, 1, 1, 3, ps, r.randint(0, 2 * ps))) for _ in range(B)]
            got = book.reserve(n_new)
            jssa.pages_reserve(L, i32(n_new), table, ref, lens, src, dst, ws)
            if got is None:
                assert jssa.read_device_status(ws) == (5, jssa.DEV_NO_PAGES)
                jssa.workspace_init(ws)
                refused += 1
                got = [-1] * B, [-1] * B
            assert (src.tolist(), dst.tolist()) == tuple(map(list, got))
        elif op == "fork":
            empty = [b for b in range(B) if book.lens[b] == 0]
            held = [b for b in range(B) if book.lens[b] > 0] or [b for b in range(B) if b not in empty]
            if not empty or not held:
                continue
            r.shuffle(empty)
            to = empty[:r.randint(1, len(empty))]
            pairs = [(r.choice(held + [-1]), b) for b in to]
            a, b = [x for x, _ in pairs], [y for _, y in pairs]
            book.fork(a, b)
            jssa.pages_fork(L, i32(a), i32(b), table, ref, lens, ws)
        elif op == "compact":
            cap = r.choice((1, 5, n_pages))
            s, t = i32([0] * cap), i32([0] * cap)
            want = book.compact(cap)
            jssa.pages_compact(L, table, ref, s, t, n_moves, ws)
            m = int(n_moves)
            assert (s[:m].tolist(), t[:m].tolist()) == want
            assert bool((s[m:] == -1).all()) and bool((t[m:] == -1).all())
        else:
            ended = [int(op == "release" and r.random() < 0.4) for _ in range(B)]
            window, sinks = (0, 0) if op == "release" else (r.choice((1, 20, ps)), r.choice((0, 4, ps + 1)))
            book.release(ended, window, sinks)
            jssa.pages_release(L, i32(ended) if op == "release" else None, window, sinks, table, ref, lens, ws)
        _same(book, table, ref, lens)
        assert jssa.read_device_status(ws)[1] == 0, (step, op)


def test_fork_skips_what_it_cannot_do():
    K = torch.zeros(8, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    book = Book(6, 2, 8, 16)
    book.reserve([20, 5, 0, 0, 0, 0])
    for src, dst in (([0], [1]), ([0], [6]), ([6], [2]), ([0], [0]), ([0], [-1]), ([0, 2], [2, 3]), ([1, 1], [4, 4])):
        table, ref, lens = _state(book)
        L = jssa.make_paged_layout(K, K, table, 1)
        ws = jssa.alloc_paged_workspace(L)
        jssa.pages_fork(L, i32(src), i32(dst), table, ref, lens, ws)
        assert jssa.read_device_status(ws)[1] == jssa.DEV_BAD_INDEX
        if dst == [4, 4]:   # the first of two takes the place
            want = Book(6, 2, 8, 16)
            want.reserve([20, 5, 0, 0, 0, 0])
            want.fork([1], [4])
            _same(want, table, ref, lens)
        else:
            _same(book, table, ref, lens)


def test_reserve_and_release_flag_bad_state():
    K = torch.zeros(8, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    book = Book(3, 2, 8, 16)
    book.reserve([20, 5, 0])
    table, ref, lens = _state(book)
    L = jssa.make_paged_layout(K, K, table, 1)
    ws = jssa.alloc_paged_workspace(L)
    src, dst = i32([7] * 3), i32([7] * 3)
    jssa.pages_reserve(L, i32([-4, 2, 16]), table, ref, lens, src, dst, ws)
    assert jssa.read_device_status(ws)[1] == jssa.DEV_BAD_SEQ_LEN
    book.reserve([0, 2, 16])
    _same(book, table, ref, lens)
    jssa.workspace_init(ws)
    table[1, 0] = -1   # the page that the next token would go to
    jssa.pages_reserve(L, i32([0, 1, 1]), table, ref, lens, src, dst, ws)
    assert jssa.read_device_status(ws)[1] == jssa.DEV_NO_PAGES
    assert src.tolist() == dst.tolist() == [-1] * 3 and lens.tolist() == book.lens
    jssa.workspace_init(ws)
    table[1, 0] = 8    # no page of the pool
    ref[table[0, 0]] = 0
    jssa.pages_release(L, i32([1, 1, 0]), 0, 0, table, ref, lens, ws)
    assert jssa.read_device_status(ws)[1] == jssa.DEV_BAD_INDEX
    assert table[:2].tolist() == [[-1, -1], [-1, -1]] and bool((ref >= 0).all())


@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("d,Hkv,page", [(64, 1, 16), (128, 3, 48), (256, 8, 256)])
def test_copy_moves_whole_pages_and_no_other(d, Hkv, page, nhd):
    n_pages = 30
    K, V = pool(n_pages, Hkv, page, d, nhd, 0.0), pool(n_pages, Hkv, page, d, not nhd, 0.0)
    K.normal_()
    V.normal_()
    L = jssa.make_paged_layout(K, V, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), Hkv)
    ws = jssa.alloc_paged_workspace(L)
    order = torch.randperm(n_pages).tolist()
    src, dst = order[:11], order[11:22]
    src[3] = -1
    dst[5] = -1
    for count in (None, 7, 0, 100, -3):
        k, v = K.clone(), V.clone()
        for a, b in list(zip(src, dst))[:None if count is None else max(0, count)]:
            if a >= 0 and b >= 0:
                k[b], v[b] = K[a], V[a]
        jssa.pages_copy(L, K, V, i32(src), i32(dst), None if count is None else i32([count]), ws)
        assert jssa.read_device_status(ws)[1] == 0
        assert torch.equal(K, k) and torch.equal(V, v)
    jssa.pages_copy(L, K, V, i32([0, n_pages, 1]), i32([n_pages, 2, 3]), None, ws)
    assert jssa.read_device_status(ws)[1] == jssa.DEV_BAD_INDEX
    k[3], v[3] = K[1], V[1]
    assert torch.equal(K, k) and torch.equal(V, v)


# --------------------------------------------------------------------------- together
def _serve(d, G, window, sinks, seed):
    """Prompts in chunks, forks, tokens one by one, ends and compaction over one cache; every
    attention is compared with the formula over rows kept apart, sequence by sequence."""
    r = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, Hkv, page, n_pages, mp = 9, 2, 16, 150, 40
    Hq = Hkv * G
    K, V = pool(n_pages, Hkv, page, d, False), pool(n_pages, Hkv, page, d, False)
    table, ref, lens = torch.full((B, mp), -1, dtype=torch.int32, device="cuda"), i32([0] * n_pages), i32([0] * B)
    L = jssa.make_paged_layout(K, V, table, Hq, jssa.OUT_F32)
    ws = jssa.alloc_paged_workspace(L, 200)
    src, dst, n_moves = i32([0] * B), i32([0] * B), i32([0])
    msrc, mdst = i32([0] * n_pages), i32([0] * n_pages)
    rows = [(torch.zeros(0, Hkv, d, dtype=torch.bfloat16, device="cuda"),) * 2 for _ in range(B)]

    def step(n_new):
        begin = [0]
        for x in n_new:
            begin.append(begin[-1] + x)
        x = torch.randn(begin[-1], Hq + 2 * Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
        q, kn, vn = x.split((Hq, Hkv, Hkv), 1)
        qb = i32(begin)
        jssa.pages_reserve(L, i32(n_new), table, ref, lens, src, dst, ws)
        jssa.pages_copy(L, K, V, src, dst, None, ws)
        jssa.paged_append_kv(L, kn, vn, K, V, table, qb, lens, ws)
        O = torch.empty(begin[-1], Hq, d, device="cuda")
        jssa.paged_attn(L, q, K, V, table, qb, max(n_new), lens, window, sinks, d ** -0.5, O, None, ws)
        assert jssa.read_device_status(ws)[1] == 0
        for b in range(B):
            lo, hi = begin[b], begin[b + 1]
            if lo == hi:
                continue
            rows[b] = tuple(torch.cat([o, n[lo:hi]]) for o, n in zip(rows[b], (kn, vn)))
            n = rows[b][0].shape[0]
            want, a, _ = attention64(q[lo:hi], rows[b][0].transpose(0, 1), rows[b][1].transpose(0, 1),
                                     torch.arange(n - (hi - lo), n, device="cuda"), torch.arange(n, device="cuda"),
                                     window, sinks, d ** -0.5)
            assert bool(((O[lo:hi].double() - want).abs() <= P_TOL * a + 2.0 ** -24 * want.abs()).all()), b

    step([130, 77, 0, 0, 0, 0, 0, 0, 0])
    step([61, 160, 0, 0, 0, 0, 0, 0, 16])
    for a, b in ((0, 2), (0, 3), (1, 4), (1, 5), (0, 6)):
        rows[b] = rows[a]
    jssa.pages_fork(L, i32([0, 0, 1, 1, 0]), i32([2, 3, 4, 5, 6]), table, ref, lens, ws)
    for turn in range(6):
        step([1, 1, 1, 0 if turn < 3 else 2, 1, 1, 1, 0, 1])
        if turn == 2:
            ended = [0, 0, 1, 0, 0, 1, 0, 0, 0]
            for b in (2, 5):
                rows[b] = tuple(x[:0] for x in rows[b])
            jssa.pages_release(L, i32(ended), window, sinks, table, ref, lens, ws)
            jssa.pages_compact(L, table, ref, msrc, mdst, n_moves, ws)
            jssa.pages_copy(L, K, V, msrc, mdst, n_moves, ws)
            held = ref.tolist()
            assert 0 not in held[:sum(x > 0 for x in held)]
            step([0, 0, 40, 0, 0, 0, 0, 7, 0])
    jssa.pages_release(L, i32([1] * B), 0, 0, table, ref, lens, ws)
    torch.cuda.synchronize()
    assert not ref.any() and not lens.any() and bool((table == -1).all())


@pytest.mark.parametrize("d,G,window,sinks", [(128, 4, 0, 0), (64, 3, 50, 4), (256, 2, 64, 0)])
def test_a_serving_run(d, G, window, sinks):
    _serve(d, G, window, sinks, 7)


def test_contiguous_cache_is_filled_and_read_as_a_pool():
    # prompt into a contiguous cache through the paged calls, then the library's dense decode and
    # the paged attention of one token over the same cache
    B, Hkv, Hq, d, T = 3, 2, 8, 128, 320
    K = torch.zeros(B, Hkv, T, d, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    L = jssa.make_paged_layout(K, V, table, Hq)
    ws = jssa.alloc_paged_workspace(L, 1)
    lens = [300, 17, 128]
    begin = [0, 300, 317, 445]
    x = torch.randn(445, 2 * Hkv, d, device="cuda").to(torch.bfloat16)
    jssa.paged_append_kv(L, x[:, :Hkv], x[:, Hkv:], K, V, table, i32(begin), i32(lens), ws)
    q = torch.randn(B, Hq, d, device="cuda").to(torch.bfloat16)
    O1, O2 = torch.empty(2, B, Hq, d, device="cuda")
    jssa.paged_attn(L, q, K, V, table, i32([0, 1, 2, 3]), 1, i32(lens), 0, 0, d ** -0.5, O1, None, ws)
    Kp = torch.zeros(B, Hkv, T, 16, dtype=torch.bfloat16, device="cuda")
    L2 = jssa.make_layout(K, V, Kp, Hq, 16)
    jssa.dense_decode(L2, q, K, V, i32(lens), 0, d ** -0.5, O2, None, jssa.alloc_workspace(L2, 16))
    for b in range(B):
        assert torch.equal(K[b, :, :lens[b]], x[begin[b]:begin[b + 1], :Hkv].transpose(0, 1))
        want, a, _ = attention64(q[b:b + 1], K[b, :, :lens[b]], V[b, :, :lens[b]], torch.tensor([lens[b] - 1]).cuda(),
                                 torch.arange(lens[b], device="cuda"), 0, 0, d ** -0.5)
        for o in (O1, O2):
            assert bool(((o[b:b + 1].double() - want).abs() <= P_TOL * a + 2.0 ** -24 * want.abs()).all())


def test_captured_and_replayed_and_on_another_stream():
    p = Problem([700, 1300, 45], [130, 1, 45], page=32, window=400, sinks=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    p.run()
    torch.cuda.synchronize()
    want = p.O.clone()
    with torch.cuda.graph(graph, stream=side):
        p.run()
    for _ in range(3):
        p.O.fill_(-777.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.O, want)
    p.check()
    # two graphs that share a workspace, replayed in turn
    q = Problem([3000, 10], [1, 10], page=32, window=400, sinks=4, seed=9)
    q.ws = p.ws = max(p.ws, q.ws, key=len)
    q.run()
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2, stream=side):
        q.run()
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph(), stream=side):
        p.run()
    for _ in range(3):
        graph.replay()
        graph2.replay()
    p.check()
    q.check()
    # two calls at once, each with a workspace of its own
    a, b = Problem([5000], [1], seed=2), Problem([900], [300], seed=3)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(stream=s1)
        b.run(stream=s2)
    a.check()
    b.check()


def test_page_operations_captured():
    K = torch.zeros(40, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    book = Book(4, 6, 40, 16)
    book.reserve([20, 33, 0, 0])
    table, ref, lens = _state(book)
    start = table.clone(), ref.clone(), lens.clone()
    L = jssa.make_paged_layout(K, K.clone(), table, 1)
    V = K.clone()
    ws = jssa.alloc_paged_workspace(L)
    src, dst, fs, fd, add = i32([0] * 4), i32([0] * 4), i32([0, 1]), i32([3, 2]), i32([1, 1, 1, 20])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jssa.pages_fork(L, fs, fd, table, ref, lens, ws)
        jssa.pages_reserve(L, add, table, ref, lens, src, dst, ws)
        jssa.pages_copy(L, K, V, src, dst, None, ws)
    book.fork([0, 1], [3, 2])
    book.reserve([1, 1, 1, 20])
    for _ in range(3):
        for x, y in zip((table, ref, lens), start):
            x.copy_(y)
        graph.replay()
        _same(book, table, ref, lens)
    assert jssa.read_device_status(ws)[1] == 0


def test_offsets_past_32_bits():
    # a pool of more than 2^32 elements (8.6 GB): its last pages, heads inside the rows
    Hkv, page, d = 8, 64, 128
    n_pages = (1 << 32) // (Hkv * page * d) + 3
    K, V = pool(n_pages, Hkv, page, d, True, 0.0), pool(n_pages, Hkv, page, d, False, 0.0)
    table = i32([[n_pages - 1, n_pages - 3, 0], [n_pages - 2, 1, 2]])
    lens, begin = [150, 70], [0, 100, 101]
    rows = torch.randn(101, 2 * Hkv, d, device="cuda").to(torch.bfloat16)
    L = jssa.make_paged_layout(K, V, table, Hkv)
    ws = jssa.alloc_paged_workspace(L, 100)
    kn, vn = rows[:, :Hkv], rows[:, Hkv:]
    jssa.paged_append_kv(L, kn, vn, K, V, table, i32(begin), i32(lens), ws)
    O = torch.empty(101, Hkv, d, device="cuda")
    jssa.paged_attn(L, kn, K, V, table, i32(begin), 100, i32(lens), 0, 0, d ** -0.5, O, None, ws)
    jssa.pages_copy(L, K, V, i32([n_pages - 1]), i32([n_pages - 4]), None, ws)
    assert jssa.read_device_status(ws)[1] == 0
    for b in range(2):
        lo, hi, n = begin[b], begin[b + 1], lens[b]
        k, v = torch.zeros(2, Hkv, n, d, dtype=torch.bfloat16, device="cuda")
        k[:, n - (hi - lo):], v[:, n - (hi - lo):] = kn[lo:hi].transpose(0, 1), vn[lo:hi].transpose(0, 1)
        want, a, _ = attention64(kn[lo:hi], k, v, torch.arange(n - (hi - lo), n, device="cuda"),
                                 torch.arange(n, device="cuda"), 0, 0, d ** -0.5)
        assert bool(((O[lo:hi].double() - want).abs() <= P_TOL * a + 2.0 ** -24 * want.abs()).all())
    assert torch.equal(K[n_pages - 4], K[n_pages - 1]) and torch.equal(V[n_pages - 4], V[n_pages - 1])
    assert bool(K[n_pages - 4].any())
