"""How exactly the paged attention weighs its rows.

The bounds of test_gpu_paged.py leave room for probabilities rounded to bf16 everywhere.  These are
as narrow as the arithmetic: which rows a query sees is checked row by row with equal logits, and
where probabilities go into the product with V in two bf16 parts, a probability is bounded by 2^-16.
"""
from __future__ import annotations

import pytest
import torch

import token_level_sparse_jssa_b200 as jssa
from tests._paged import seen_mask
from tests.test_gpu_paged import Problem

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])


def _seen(p, b):
    """[queries, seen tokens] of sequence b, as a mask."""
    return seen_mask(p.pos[b], p.t[b], p.window, p.sinks)


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
