"""How exactly the paged attention weighs its rows.

The bounds of test_gpu_paged.py leave room for probabilities rounded to bf16 everywhere.  These are
as narrow as the arithmetic: which rows a query sees is checked row by row with equal logits, and
where probabilities go into the product with V in two bf16 parts, a probability is bounded by 2^-16.
"""
from __future__ import annotations

import pytest
import torch

import token_level_sparse_jssa_b200 as jssa
from tests._paged import attention64, seen_mask
from tests.test_gpu_paged import CASES, Problem

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])


def _fill(p, pool, b, rows):
    """Writes rows [T, Hkv, d] as sequence b's seen tokens p.t[b] into a pool."""
    t = p.t[b]
    if len(t):
        pool[p.table[b].long()[t // p.page], :, t % p.page] = rows.to(torch.bfloat16)


def _seen(p, b):
    """[queries, seen tokens] of sequence b, as a mask."""
    return seen_mask(p.pos[b], p.t[b], p.window, p.sinks)


# --------------------------------------------------------------------------- which rows are seen
@BOTH
@pytest.mark.parametrize("kw", CASES)
def test_every_seen_row_counts_once(kw, out):
    # Equal logits (Q = 0): every p is 1, the output is the mean of the seen rows and lse = log n.  V holds whole numbers
    # from -127 to 127 but 0, whose sums are exact in fp32 (at most 16,000 rows: under 2^21), so in fp32 the
    # output is off by the reciprocal's and the product's rounding, and a lost or doubled row moves it by more:
    # by 1/n at least, against 2^-23 |mean| with |mean| <= 127 and n <= 16,000.  In bf16, 2^-8 of the rounding, 2^-15
    # of the row sum's exponentials (7.5e-5 on one in 16), and the row test below tells single rows.
    p = Problem(**kw, out=out)
    p.Q.zero_()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    v = []
    for b in range(len(p.lens)):
        x = torch.randint(1, 128, (len(p.t[b]), p.Hkv, p.d), generator=g, device="cuda")
        x *= 1 - 2 * torch.randint(0, 2, x.shape, generator=g, device="cuda")
        _fill(p, p.V, b, x)
        v.append(x.double())
    p.run()
    torch.cuda.synchronize()
    assert jssa.read_device_status(p.ws)[1] == 0
    tol, lse_tol = (2.0 ** -22.9, 2.0 ** -21) if out == torch.float32 else (2.0 ** -8 + 2.0 ** -15, 2.0 ** -15)
    for b in range(len(p.lens)):
        lo, hi = p.begin[b], p.begin[b + 1]
        if lo == hi:
            continue
        m = _seen(p, b).double()
        n = m.sum(1)
        want = torch.einsum("qt,thd->qhd", m, v[b]) / n[:, None, None]
        want = want.repeat_interleave(p.Hq // p.Hkv, 1)
        err = (p.O[lo:hi].double() - want).abs()
        assert bool((err <= tol * want.abs()).all()), (b, float((err / want.abs().clamp(min=1e-30)).max()))
        lse = n.log()[:, None]
        assert bool(((p.lse[lo:hi].double() - lse).abs() <= lse_tol * (1 + lse)).all()), b


@BOTH
@pytest.mark.parametrize("kw", CASES)
def test_each_edge_row_is_seen_by_its_queries_alone(kw, out):
    # Column e of V is 64 in one row alone, in turn at the ends of pages, tiles, windows, sinks and sequences: the output's
    # column is 64 / n for the queries that see that row and exactly 0 for the others.
    p = Problem(**kw, out=out)
    p.Q.zero_()
    rows = []
    for b in range(len(p.lens)):
        t = p.t[b]
        edge = {0, 1, p.lens[b] - 1, p.lens[b] - p.nq[b], p.lens[b] - p.nq[b] - 1, p.sinks - 1, p.sinks}
        for q in (p.lens[b] - p.nq[b], p.lens[b] - 1):
            edge |= {q - p.window, q - p.window + 1, q - p.window + 2}
        for unit in (p.page, 64, 128):
            for x in (p.lens[b] // 2, p.lens[b] - p.nq[b], p.lens[b] - 1):
                edge |= {x // unit * unit - 1, x // unit * unit}
        at = [i for i, x in enumerate(t.tolist()) if x in edge]
        at = (at * p.d)[:p.d] if len(at) < p.d else at[:p.d]
        x = torch.zeros(len(t), p.Hkv, p.d, device="cuda")
        if at:
            x[torch.tensor(at), :, torch.arange(p.d)] = 64.0
        _fill(p, p.V, b, x)
        rows.append(at)
    p.run()
    torch.cuda.synchronize()
    assert jssa.read_device_status(p.ws)[1] == 0
    tol = 2.0 ** -22.9 if out == torch.float32 else 2.0 ** -8 + 2.0 ** -15
    for b in range(len(p.lens)):
        lo, hi = p.begin[b], p.begin[b + 1]
        if lo == hi:
            continue
        m = _seen(p, b).double()
        want = (64.0 * m[:, rows[b]] / m.sum(1, keepdim=True))[:, None, :]
        assert bool(((p.O[lo:hi].double() - want).abs() <= tol * want).all()), b


# --------------------------------------------------------------------------- probabilities
def _two_level(p):
    """Every 16th token has logit 0 and the others log(0.50193), which lies between two bf16 values (0.5 is 3.9e-3 off), so
    that each key warp and tile keeps its maximum at 0; the values cancel, so that the
    output is small beside sum p|v| and its own rounding hides nothing."""
    p.scale = 1.0
    p.Q.zero_()
    p.Q[..., 0] = 1.0
    for b in range(len(p.lens)):
        top = (p.t[b] % 16 == 0)
        k = torch.zeros(len(p.t[b]), p.Hkv, p.d, device="cuda")
        k[:, :, 0] = torch.where(top, 0.0, -1.0)[:, None]
        v = torch.where(top, -7.53125, 1.0)[:, None, None].expand_as(k)
        _fill(p, p.K, b, k)
        _fill(p, p.V, b, v)
        p.k64[b], p.v64[b] = (x.to(torch.bfloat16).transpose(0, 1) for x in (k, v))
    p.scale = 0.68929454   # -log(0.50193)


def _check_two_level(p, two):
    torch.cuda.synchronize()
    assert jssa.read_device_status(p.ws)[1] == 0
    for b in range(len(p.lens)):
        lo, hi = p.begin[b], p.begin[b + 1]
        if lo == hi:
            continue
        want, a, _ = attention64(p.Q[lo:hi], p.k64[b], p.v64[b], p.pos[b], p.t[b], p.window, p.sinks, p.scale)
        # p: two parts 2^-16, the exponential, the logit's and the scale's rounding 2^-20; sums of at most
        # lens[b] terms in fp32, above and below the line.  One part: 2^-8 in place of 2^-16, and 7.5e-5 of the cubic.
        tol = (2.0 ** -16 if two(b) else 2.0 ** -8 + 2.0 ** -13) + 2.0 ** -20 + 2 * p.lens[b] * 2.0 ** -24
        tol = tol * a + (2.0 ** -8 if p.out == torch.bfloat16 else 2.0 ** -24) * want.abs()
        err = (p.O[lo:hi].double() - want).abs()
        assert bool((err <= tol).all()), (b, float((err / a).max()))


@BOTH
@pytest.mark.parametrize("kw", [
    dict(lens=[600, 31], nq=[1, 1], G=4), dict(lens=[600, 17], nq=[4, 3], d=64, G=8, Hkv=1),
    dict(lens=[500], nq=[2], d=256, G=4, page=64), dict(lens=[700, 90], nq=[30, 5], G=4, window=300, sinks=5),
    dict(lens=[700, 90], nq=[16, 1], G=8, d=64), dict(lens=[700, 90], nq=[64, 9], G=2, d=256),
    dict(lens=[300], nq=[1], G=128, Hkv=1),
])
def test_few_rows_keep_sixteen_bits_of_a_probability(kw, out):
    p = Problem(**kw, out=out)
    _two_level(p)
    p.run()
    _check_two_level(p, lambda b: True)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_fp32_outputs_keep_sixteen_bits_of_a_probability(d):
    p = Problem([700, 90, 300], [300, 1, 5], d=d, G=4, out=torch.float32)
    _two_level(p)
    p.run()
    _check_two_level(p, lambda b: True)


@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("d,G", [(64, 4), (128, 4), (256, 2), (128, 16), (64, 128)])
def test_precision_is_a_sequences_own(d, G, window):
    # sequences of at most 128 rows per KV head beside a prompt chunk, and under a generous bound
    few = 128 // G
    p = Problem([700, 600, 450, 90, 500], [200, 1, few, min(3, few), few + 1], d=d, Hkv=1, G=G, window=window, sinks=3)
    _two_level(p)
    p.run()
    _check_two_level(p, lambda b: b in (1, 2, 3))
    p = Problem([600, 90], [1, few], d=d, Hkv=1, G=G, window=window, sinks=3)
    p.max_q = 5000
    p.ws = jssa.alloc_paged_workspace(p.L, p.max_q)
    _two_level(p)
    p.run()
    _check_two_level(p, lambda b: True)
    if G == 4:   # cut over the whole GPU
        p = Problem([700, 9000], [200, 1], d=d, Hkv=1, G=G, window=0)
        _two_level(p)
        p.run()
        _check_two_level(p, lambda b: b == 1)


# --------------------------------------------------------------------------- hidden rows
@BOTH
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_hidden_values_of_any_size_change_nothing(d, window, out):
    # values of 6e36 (44 of them add up to less than the largest fp32) in rows that some queries of a tile see and
    # others do not: the others' outputs keep every bit
    T, first = 400, 70
    p = Problem([T, 150], [T, 60], d=d, Hkv=2, G=2, window=window, sinks=2, out=out)
    p.Q.zero_()
    p.run()
    want, lse = p.O.clone(), p.lse.clone()
    huge = torch.arange(T, device="cuda") % 32 >= 28   # a few in each 32 keys, from token `first` on
    huge[:first] = False
    at = p.t[0][huge]
    p.V[p.table[0].long()[at // p.page], :, at % p.page] = 6e36
    p.O.fill_(-777.0)
    p.run()
    torch.cuda.synchronize()
    assert jssa.read_device_status(p.ws)[1] == 0
    clean = ~(_seen(p, 0) & huge).any(1)
    assert int(clean.sum()) >= first and bool(torch.equal(p.lse, lse))
    assert torch.equal(p.O[:T][clean], want[:T][clean])
    assert torch.equal(p.O[T:], want[T:])
    assert bool(torch.isfinite(p.O).all())
