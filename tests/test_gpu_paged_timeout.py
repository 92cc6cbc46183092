"""The paged attention's bounded waits give up, report and return.

The library's one-shot test request withholds something in the first CTA: a copy of V in the kernel for prompts, a
warp's arrival in the one for few rows.  Everything in that CTA that waits for it, or for what depends on it, gives
up after a second; copies under way land, matrix products are drained, tensor memory is freed.
Nothing faults or hangs: the call returns with the timeout in its status, and with a workspace that was
initialised again the next call gives every bit of a clean run.
"""
from __future__ import annotations

import pytest
import torch

import token_level_sparse_jssa_b200 as jssa
from tests.test_gpu_paged import Problem

pytestmark = pytest.mark.gpu

LIMIT_US = 2000   # of the selection kernels; the paged ones have their own
TIMEOUT = 6   # JSSA_ERR_TIMEOUT


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", [   # enough work that the first CTA has a tile
    # few rows: cut items and whole ones, one and two row tiles
    dict(lens=[2048] * 8, nq=[1] * 8, Hkv=8), dict(lens=[60] * 200, nq=[1] * 200),
    dict(lens=[1500] * 8, nq=[1] * 8, d=256, Hkv=8, G=2, page=64, window=1024, sinks=4),
    dict(lens=[900, 400] * 10, nq=[17, 20] * 10, d=64, Hkv=8, G=1, window=700, sinks=20, page=48),
    # prompts: pairs of query tiles and single ones, cut items of many rows and of few, edge tiles of both kinds
    dict(lens=[1000, 300, 1200] * 3, nq=[400, 3, 130] * 3, Hkv=4, page=64),
    dict(lens=[800] * 4, nq=[800] * 4, d=256, Hkv=4, G=1, window=200, sinks=70),
    dict(lens=[1500, 77] * 4, nq=[700, 77] * 4, d=64, G=8, window=600, sinks=5, page=32),
    dict(lens=[2000] * 8, nq=[8] * 8, G=4, Hkv=8), dict(lens=[9000], nq=[100], Hkv=1, G=1),
    dict(lens=[30] * 100, nq=[30] * 100, G=4),
])
def test_a_withheld_copy_is_reported_and_the_next_call_is_clean(kw, out):
    p = Problem(**kw, out=out)
    p.run()
    p.check()
    want, lse = p.O.clone(), p.lse.clone()
    jssa.arm_withheld_copy(p.ws, LIMIT_US)
    p.run()                                           # returns
    code, flags = jssa.read_device_status(p.ws)       # synchronises
    assert code == TIMEOUT and flags == jssa.DEV_TIMEOUT
    jssa.workspace_init(p.ws)
    for _ in range(2):
        p.O.fill_(-777.0)
        p.lse.fill_(-777.0)
        p.run()
        p.check()
        assert torch.equal(p.O, want) and torch.equal(p.lse, lse)


@pytest.mark.parametrize("max_q", [1, 200])
def test_a_request_without_work_to_withhold_is_spent(max_q):
    p = Problem([0, 0], [0, 0], tail=3)
    q = Problem([2000] * 8, [max_q] * 8, Hkv=8)
    p.max_q, p.ws = max_q, q.ws
    jssa.arm_withheld_copy(q.ws, LIMIT_US)
    p.run()
    p.check()
    q.run()
    q.check()
