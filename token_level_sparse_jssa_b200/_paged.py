"""ctypes binding of the paged-cache entry points of libjssa.so (include/jssa.h).

Argument marshalling as in _binding.py.  The shapes, types and device of every tensor are
checked against the layout here, because the C ABI takes bare pointers.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _binding as _b
from ._binding import OUT_BF16, OUT_F32, _check, _stream, load, workspace_init


class PagedLayout(C.Structure):
    _fields_ = [("B", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("d", C.c_int32), ("page_size", C.c_int32),
                ("n_pages", C.c_int32), ("max_pages", C.c_int32), ("out_dtype", C.c_int32),
                ("k_stride", C.c_int64 * 3), ("v_stride", C.c_int64 * 3)]


def _signatures():
    vp, i32, i64, f32, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
    LP = C.POINTER(PagedLayout)
    end = [vp, sz, vp]   # workspace, its bytes, stream
    return {
        "jssa_paged_workspace_size": (C.c_int, [LP, i32, C.POINTER(sz)]),
        "jssa_paged_append_kv": (C.c_int, [LP, vp, vp, i64, i64, vp, vp, vp, vp, vp] + end),
        "jssa_paged_attn": (C.c_int, [LP, vp, i64, i64, i32, vp, vp, vp, vp, vp, i32, i32, f32, vp, vp] + end),
        "jssa_pages_fork": (C.c_int, [LP, vp, vp, i32, vp, vp, vp] + end),
        "jssa_pages_reserve": (C.c_int, [LP, vp, vp, vp, vp, vp, vp] + end),
        "jssa_pages_release": (C.c_int, [LP, vp, i32, i32, vp, vp, vp] + end),
        "jssa_pages_compact": (C.c_int, [LP, vp, vp, vp, vp, i32, vp] + end),
        "jssa_pages_copy": (C.c_int, [LP, vp, vp, vp, vp, i32, vp] + end),
    }


_b.SIGNATURE_SOURCES.append(_signatures)


def _dev(t, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: device tensor expected")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{what} is on {t.device}, not on the current device")
    return t


def _i32(t, shape, what):
    """Pointer of a contiguous int32 device tensor of the given shape (-1: any length)."""
    _dev(t, what)
    if t.dtype != torch.int32 or t.dim() != len(shape) or any(w not in (-1, n) for w, n in zip(shape, t.shape)):
        raise ValueError(f"{what}: int32 tensor of shape {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: contiguous tensor expected")
    return t.data_ptr()


def _pool(L, t, strides, what):
    _dev(t, what)
    if t.dtype != torch.bfloat16 or tuple(t.shape) != (L.n_pages, L.Hkv, L.page_size, L.d) or t.stride(3) != 1:
        raise ValueError(f"{what}: bfloat16 pool [n_pages, Hkv, page_size, d] of the layout expected")
    if any(n > 1 and a != b for n, a, b in zip(t.shape, t.stride(), strides)):
        raise ValueError(f"{what}: strides {t.stride()} differ from the layout's")
    return t.data_ptr()


def _rows(t, heads, d, what):
    """(pointer, row stride) of packed token rows [n, heads, d], each row's heads contiguous."""
    _dev(t, what)
    if t.dtype != torch.bfloat16 or t.dim() != 3 or tuple(t.shape[1:]) != (heads, d):
        raise ValueError(f"{what}: bfloat16 rows [n, {heads}, {d}] expected, got {t.dtype} {tuple(t.shape)}")
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"{what}: the heads of a row must be contiguous")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else heads * d)


def _ws(ws):
    if ws is None:
        return None, 0
    return _dev(ws, "ws").data_ptr(), ws.numel() * ws.element_size()


def _book(L, page_table, ref_count, seq_lens):
    return (_i32(page_table, (L.B, L.max_pages), "page_table"), _i32(ref_count, (L.n_pages,), "ref_count"),
            _i32(seq_lens, (L.B,), "seq_lens"))


def make_paged_layout(K: torch.Tensor, V: torch.Tensor, page_table: torch.Tensor, Hq: int,
                      out_dtype: int = OUT_F32) -> PagedLayout:
    """Layout from pools K and V [n_pages, Hkv, page_size, d] (any strides with a contiguous last
    dimension) and the page table [B, max_pages].  A contiguous cache [B, Hkv, T_cap, d] is a
    pool of B pages; its table is torch.arange(B, dtype=torch.int32)[:, None]."""
    if K.dim() != 4 or K.shape != V.shape or page_table.dim() != 2:
        raise ValueError("K and V [n_pages, Hkv, page_size, d] and page_table [B, max_pages] expected")
    L = PagedLayout()
    L.n_pages, L.Hkv, L.page_size, L.d = K.shape
    L.B, L.max_pages = page_table.shape
    L.Hq, L.out_dtype = Hq, out_dtype
    for i in range(3):
        L.k_stride[i] = K.stride(i)
        L.v_stride[i] = V.stride(i)
    return L


def paged_workspace_size(L: PagedLayout, max_q_len: int = 0) -> int:
    n = C.c_size_t(0)
    _check("jssa_paged_workspace_size", load().jssa_paged_workspace_size(C.byref(L), max_q_len, C.byref(n)))
    return n.value


def alloc_paged_workspace(L: PagedLayout, max_q_len: int = 0, device=None) -> torch.Tensor:
    """Caller-side allocation of the paged calls' workspace, zeroed; max_q_len as in paged_attn."""
    ws = torch.empty(paged_workspace_size(L, max_q_len), dtype=torch.uint8, device=device or "cuda")
    workspace_init(ws)
    return ws


def paged_append_kv(L, K_new, V_new, K, V, page_table, q_begin, seq_lens, ws, stream=None):
    """Write the newest tokens' rows K_new, V_new [n_tokens, Hkv, d] into their pages."""
    k, ks = _rows(K_new, L.Hkv, L.d, "K_new")
    v, vs = _rows(V_new, L.Hkv, L.d, "V_new")
    if K_new.shape[0] != V_new.shape[0] or ks != vs:
        raise ValueError("K_new and V_new must have the same rows and row stride")
    w, n = _ws(ws)
    _check("jssa_paged_append_kv", load().jssa_paged_append_kv(
        C.byref(L), k, v, ks, K_new.shape[0], _pool(L, K, L.k_stride, "K"), _pool(L, V, L.v_stride, "V"),
        _i32(page_table, (L.B, L.max_pages), "page_table"), _i32(q_begin, (L.B + 1,), "q_begin"),
        _i32(seq_lens, (L.B,), "seq_lens"), w, n, _stream(stream)))


def paged_attn(L, Q, K, V, page_table, q_begin, max_q_len: int, seq_lens, window: int, n_sinks: int, sm_scale: float,
               O, lse=None, ws=None, stream=None):
    """Causal attention of the newest tokens Q [n_tokens, Hq, d] over their sequences' pages, with
    an optional sliding window (window > 0) and n_sinks first tokens that stay visible."""
    q, qs = _rows(Q, L.Hq, L.d, "Q")
    rows = (Q.shape[0], L.Hq)
    _dev(O, "O")
    if tuple(O.shape) != rows + (L.d,) or not O.is_contiguous() or \
            O.dtype != (torch.bfloat16 if L.out_dtype == OUT_BF16 else torch.float32):
        raise ValueError("O: contiguous [n_tokens, Hq, d] of the layout's output type expected")
    if lse is not None:
        _dev(lse, "lse")
        if tuple(lse.shape) != rows or not lse.is_contiguous() or lse.dtype != torch.float32:
            raise ValueError("lse: contiguous float32 [n_tokens, Hq] expected")
    w, n = _ws(ws)
    _check("jssa_paged_attn", load().jssa_paged_attn(
        C.byref(L), q, qs, Q.shape[0], max_q_len, _pool(L, K, L.k_stride, "K"), _pool(L, V, L.v_stride, "V"),
        _i32(page_table, (L.B, L.max_pages), "page_table"), _i32(q_begin, (L.B + 1,), "q_begin"),
        _i32(seq_lens, (L.B,), "seq_lens"), window, n_sinks, sm_scale, O.data_ptr(),
        lse.data_ptr() if lse is not None else None, w, n, _stream(stream)))


def pages_fork(L, src, dst, page_table, ref_count, seq_lens, ws, stream=None):
    """Sequence dst[i] (empty) becomes a copy of sequence src[i] that shares its pages."""
    s = _i32(src, (-1,), "src")
    w, n = _ws(ws)
    _check("jssa_pages_fork", load().jssa_pages_fork(
        C.byref(L), s, _i32(dst, (src.shape[0],), "dst"), src.shape[0], *_book(L, page_table, ref_count, seq_lens),
        w, n, _stream(stream)))


def pages_reserve(L, n_new, page_table, ref_count, seq_lens, copy_src, copy_dst, ws, stream=None):
    """Room for n_new[b] more tokens of every sequence, added to seq_lens; copy_src/copy_dst [B]
    name the shared pages to copy (pages_copy) before the append."""
    w, n = _ws(ws)
    _check("jssa_pages_reserve", load().jssa_pages_reserve(
        C.byref(L), _i32(n_new, (L.B,), "n_new"), *_book(L, page_table, ref_count, seq_lens),
        _i32(copy_src, (L.B,), "copy_src"), _i32(copy_dst, (L.B,), "copy_dst"), w, n, _stream(stream)))


def pages_release(L, ended, window: int, n_sinks: int, page_table, ref_count, seq_lens, ws, stream=None):
    """Give up all pages of the sequences with ended[b] != 0 and, with window > 0, the others' pages
    behind their last `window` tokens that hold none of the first n_sinks."""
    e = _i32(ended, (L.B,), "ended") if ended is not None else None
    w, n = _ws(ws)
    _check("jssa_pages_release", load().jssa_pages_release(
        C.byref(L), e, window, n_sinks, *_book(L, page_table, ref_count, seq_lens), w, n, _stream(stream)))


def pages_compact(L, page_table, ref_count, src, dst, n_moves, ws, stream=None):
    """Move the pages in use to the front of the pool (at most len(src) of them): the table and the
    counts now, the rows with pages_copy(..., src, dst, n_moves)."""
    s = _i32(src, (-1,), "src")
    w, n = _ws(ws)
    _check("jssa_pages_compact", load().jssa_pages_compact(
        C.byref(L), _i32(page_table, (L.B, L.max_pages), "page_table"), _i32(ref_count, (L.n_pages,), "ref_count"),
        s, _i32(dst, (src.shape[0],), "dst"), src.shape[0], _i32(n_moves, (1,), "n_moves"), w, n, _stream(stream)))


def pages_copy(L, K, V, src, dst, count=None, ws=None, stream=None):
    """Copy page src[i] over page dst[i] in both pools, for every entry or the first count[0];
    negative entries are skipped."""
    s = _i32(src, (-1,), "src")
    c = _i32(count, (1,), "count") if count is not None else None
    w, n = _ws(ws)
    _check("jssa_pages_copy", load().jssa_pages_copy(
        C.byref(L), _pool(L, K, L.k_stride, "K"), _pool(L, V, L.v_stride, "V"), s,
        _i32(dst, (src.shape[0],), "dst"), src.shape[0], c, w, n, _stream(stream)))
