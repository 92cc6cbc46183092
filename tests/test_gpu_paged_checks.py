"""What the paged calls report of arguments that only the device can see."""
from __future__ import annotations

import pytest
import torch

import token_level_sparse_jssa_b200 as jssa
from tests._paged import i32, pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("begin,lens", [
    ([0, 5, 5], [20, -1]),     # no new token, and a length that cannot be
    ([0, 5, 5], [20, 33]),     # past the table's end
    ([0, 5, 2], [20, 20]),     # ends before it begins, behind rows of another sequence
    ([0, 5, 9], [20, 20]),     # begins at the end of the rows that are there
])
def test_append_reports_a_bad_sequence_that_no_row_belongs_to(begin, lens):
    K, V = pool(8, 2, 16, 64, False, 0.0), pool(8, 2, 16, 64, False, 0.0)
    table = i32([[0, 1], [2, 3]])
    rows = torch.ones(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    L = jssa.make_paged_layout(K, V, table, 2)
    ws = jssa.alloc_paged_workspace(L)
    jssa.paged_append_kv(L, rows, rows, K, V, table, i32(begin), i32(lens), ws)
    assert jssa.read_device_status(ws) == (5, jssa.DEV_BAD_SEQ_LEN)
    # the other sequence's five rows stand at 15 to 19
    assert K.sum((1, 3)).count_nonzero(1).tolist() == [1, 4, 0, 0, 0, 0, 0, 0]
    assert torch.equal(K, V)


@pytest.mark.parametrize("d,nq", [(128, [1, 1]), (128, [130, 9]), (64, [70, 3]), (256, [40, 1])])
def test_rows_behind_the_last_sequence_may_hold_anything(d, nq):
    from tests.test_gpu_paged import Problem
    p = Problem([700, 300], nq, d=d, G=2, page=32, tail=140)
    p.Q[p.begin[-1]:] = float("nan")
    p.run()
    p.check()
    new = torch.full((p.n, p.Hkv, d), float("inf"), dtype=torch.bfloat16, device="cuda")
    new[:p.begin[-1]] = 1.0
    K, V = p.K.clone(), p.V.clone()
    jssa.paged_append_kv(p.L, new, new, K, V, p.table, p.q_begin, p.seq_lens, p.ws)
    assert jssa.read_device_status(p.ws) == (0, 0)
    assert not bool(K.isinf().any()) and not bool(V.isinf().any())
    assert int((K == 1.0).all(-1).sum()) == sum(nq) * p.Hkv
