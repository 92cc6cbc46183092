"""Limits of the paged layouts and what the binding refuses of a workspace, on the CPU."""
import ctypes as C

import pytest
import torch

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from token_level_sparse_jssa_b200 import build
    build.build()
    from token_level_sparse_jssa_b200 import _binding
    return _binding.load()


def _layout(Hkv, page, d, max_pages=1):
    from token_level_sparse_jssa_b200 import PagedLayout
    L = PagedLayout()
    L.B, L.Hq, L.Hkv, L.d, L.page_size, L.n_pages, L.max_pages = 1, Hkv, Hkv, d, page, 1, max_pages
    for st in (L.k_stride, L.v_stride):
        st[0], st[1], st[2] = Hkv * page * d, page * d, d
    return L


@pytest.mark.parametrize("Hkv,page,d,code", [
    (8, (1 << 24) - 16, 128, 0), (8, 1 << 24, 128, 2),            # 2^34 elements a page and just below
    (64, (1 << 21) - 16, 128, 0), (64, 1 << 21, 128, 2), (65, 1 << 21, 128, 2),
    (128, (1 << 21) - 16, 64, 0), (128, 1 << 21, 64, 2), (127, 1 << 21, 64, 0), (1, 1 << 26, 256, 2),
])
def test_a_page_has_less_than_two_to_the_34_elements(lib, Hkv, page, d, code):
    L = _layout(Hkv, page, d)
    # calls that return before any CUDA call, once the layout is found good
    assert lib.jssa_pages_copy(C.byref(L), None, None, None, None, 0, None, None, 0, None) == code
    assert lib.jssa_pages_fork(C.byref(L), None, None, 0, None, None, None, None, 0, None) == code


def test_a_workspace_of_repeated_or_spread_bytes_is_refused(monkeypatch):
    # its size would count bytes that are not its own
    import token_level_sparse_jssa_b200 as jssa
    from token_level_sparse_jssa_b200 import _paged
    monkeypatch.setattr(_paged, "_device", lambda: -1)      # where host tensors say they are
    monkeypatch.setattr(_paged, "_stream", lambda stream, dev: None)
    K = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 1, dtype=torch.int32)
    L = jssa.make_paged_layout(K, K, table, 1)
    none = torch.zeros(0, dtype=torch.int32)
    jssa.pages_copy(L, K, K, none, none, None, torch.zeros(4096, dtype=torch.uint8))    # nothing to copy: no CUDA call
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 30), torch.zeros(4096, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError):
            jssa.pages_copy(L, K, K, none, none, None, ws)


@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 5, 1 << 40])
def test_bounds_and_windows_past_31_bits_are_refused(value, monkeypatch):
    # an int32 argument would be cut to its low bits: a window of 2^32 + 5 tokens to one of 5
    import token_level_sparse_jssa_b200 as jssa
    from token_level_sparse_jssa_b200 import _paged
    monkeypatch.setattr(_paged, "_device", lambda: -1)
    monkeypatch.setattr(_paged, "_stream", lambda stream, dev: None)
    K = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    table, ref, lens, begin = (torch.zeros(n, dtype=torch.int32) for n in ((1, 1), 2, 1, 2))
    L = jssa.make_paged_layout(K, K, table, 1)
    Q, O, ws = torch.zeros(0, 1, 64, dtype=torch.bfloat16), torch.zeros(0, 1, 64), torch.zeros(256, dtype=torch.uint8)
    for max_q, window, sinks in ((value, 0, 0), (1, value, 0), (1, 8, value)):
        with pytest.raises(ValueError):
            jssa.paged_attn(L, Q, K, K, table, begin, max_q, lens, window, sinks, 0.1, O, None, ws)
    jssa.paged_attn(L, Q, K, K, table, begin, 1, lens, (1 << 31) - 1, 0, 0.1, O, None, ws)   # no rows: no CUDA call
    for window, sinks in ((value, 0), (8, value)):
        with pytest.raises(ValueError):
            jssa.pages_release(L, None, window, sinks, table, ref, lens, ws)
    with pytest.raises(ValueError):
        jssa.paged_workspace_size(L, value)
