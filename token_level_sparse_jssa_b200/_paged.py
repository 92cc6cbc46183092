"""ctypes binding of the paged-cache entry points of libjssa.so (include/jssa.h).

Argument marshalling as in _binding.py.  The shapes, types and device of every tensor are
checked against the layout here, because the C ABI takes bare pointers.
"""
from __future__ import annotations

import ctypes as C

import torch
from torch import Tensor

from . import _binding as _b
from ._binding import OUT_BF16, OUT_F32, _check, load, workspace_init

_I32, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32


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


# A decode step makes several of these calls, each on a few microseconds of GPU work.  So the checks
# below read every property of a tensor once, what follows from a layout's fields is derived once
# for their present values, and the wording of a refusal is left to _refuse().
class _Facts:
    __slots__ = ("fields", "heads", "pool", "k_stride", "v_stride", "table", "ref", "seq", "begin", "out")

    def __init__(self, L, fields):
        self.fields = fields
        self.heads = L.Hq, L.Hkv, L.d
        self.pool = L.n_pages, L.Hkv, L.page_size, L.d
        self.k_stride, self.v_stride = tuple(L.k_stride) + (1,), tuple(L.v_stride) + (1,)
        self.table, self.ref, self.seq, self.begin = (L.B, L.max_pages), (L.n_pages,), (L.B,), (L.B + 1,)
        self.out = _BF16 if L.out_dtype == OUT_BF16 else _F32


def _facts(L):
    fields = bytes(L)
    f = L.__dict__.get("facts")
    if f is None or f.fields != fields:
        f = L.__dict__["facts"] = _Facts(L, fields)
    return f


def _refuse(t, what, dev, expected):
    if not isinstance(t, Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: device tensor expected")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, not on the current device")
    raise ValueError(f"{what}: {expected} expected, got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")


def _device():
    return torch.cuda.current_device() if torch.cuda.is_initialized() else 0


def _stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _b._stream(stream)


def _packed(t, dtype, shape, what, dev):
    """Pointer of a contiguous device tensor of the given type and shape."""
    if not isinstance(t, Tensor) or t.get_device() != dev or t.dtype is not dtype or t.shape != shape or \
            not t.is_contiguous():
        _refuse(t, what, dev, f"contiguous {dtype} tensor of shape {shape}")
    return t.data_ptr()


def _list(t, what, dev):
    """(pointer, length) of a contiguous int32 device tensor of one dimension."""
    n = t.numel() if isinstance(t, Tensor) else 0
    return _packed(t, _I32, (n,), what, dev), n


def _pool(t, shape, strides, what, dev):
    if not isinstance(t, Tensor) or t.get_device() != dev or t.dtype is not _BF16 or t.shape != shape:
        _refuse(t, what, dev, f"bfloat16 pool {shape}")
    got = t.stride()
    if got != strides and (got[3] != 1 or any(n > 1 and x != y for n, x, y in zip(shape, got, strides))):
        _refuse(t, what, dev, f"the layout's strides {strides}")
    return t.data_ptr()


def _rows(t, heads, d, what, dev):
    """(pointer, rows, row stride) of packed token rows [n, heads, d], each row's heads contiguous."""
    if not isinstance(t, Tensor) or t.get_device() != dev or t.dtype is not _BF16 or t.dim() != 3:
        _refuse(t, what, dev, f"bfloat16 rows [n, {heads}, {d}]")
    n, h, e = t.shape
    row, head, one = t.stride()
    if h != heads or e != d or one != 1 or (head != d and heads > 1):
        _refuse(t, what, dev, f"bfloat16 rows [n, {heads}, {d}], the heads of a row contiguous,")
    return t.data_ptr(), n, (row if n > 1 else heads * d)


def _book(f, page_table, ref_count, seq_lens, dev):
    return (_packed(page_table, _I32, f.table, "page_table", dev),
            _packed(ref_count, _I32, f.ref, "ref_count", dev),
            _packed(seq_lens, _I32, f.seq, "seq_lens", dev))


def _ws(ws, dev):
    if ws is None:
        return None, 0
    if not isinstance(ws, Tensor) or ws.get_device() != dev or not ws.is_contiguous():
        _refuse(ws, "ws", dev, "contiguous workspace")
    return ws.data_ptr(), ws.nbytes


def _fits(*ints):
    """Refuses what the C ABI's int32 would silently cut (negative values are its own to refuse)."""
    if max(ints) >= 1 << 31:
        raise ValueError(f"{ints}: values below 2**31 expected")


def make_paged_layout(K: torch.Tensor, V: torch.Tensor, page_table: torch.Tensor, Hq: int,
                      out_dtype: int = OUT_F32) -> PagedLayout:
    """Layout from pools K and V [n_pages, Hkv, page_size, d] (any strides with a contiguous last
    dimension) and the page table [B, max_pages].  A contiguous cache [B, Hkv, T_cap, d] is a
    pool of B pages; its table is torch.arange(B, dtype=_I32)[:, None]."""
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
    _fits(max_q_len)
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
    dev, f = _device(), _facts(L)
    _, H, d = f.heads
    k, nk, ks = _rows(K_new, H, d, "K_new", dev)
    v, nv, vs = _rows(V_new, H, d, "V_new", dev)
    if nk != nv or ks != vs:
        raise ValueError("K_new and V_new must have the same rows and row stride")
    w, nw = _ws(ws, dev)
    code = load().jssa_paged_append_kv(
        C.byref(L), k, v, ks, nk, _pool(K, f.pool, f.k_stride, "K", dev), _pool(V, f.pool, f.v_stride, "V", dev),
        _packed(page_table, _I32, f.table, "page_table", dev),
        _packed(q_begin, _I32, f.begin, "q_begin", dev), _packed(seq_lens, _I32, f.seq, "seq_lens", dev),
        w, nw, _stream(stream, dev))
    if code:
        _check("jssa_paged_append_kv", code)


def paged_attn(L, Q, K, V, page_table, q_begin, max_q_len: int, seq_lens, window: int, n_sinks: int, sm_scale: float,
               O, lse=None, ws=None, stream=None):
    """Causal attention of the newest tokens Q [n_tokens, Hq, d] over their sequences' pages, with
    an optional sliding window (window > 0) and n_sinks first tokens that stay visible."""
    dev, f = _device(), _facts(L)
    Hq, _, d = f.heads
    _fits(max_q_len, window, n_sinks)
    q, n, qs = _rows(Q, Hq, d, "Q", dev)
    w, nw = _ws(ws, dev)
    code = load().jssa_paged_attn(
        C.byref(L), q, qs, n, max_q_len, _pool(K, f.pool, f.k_stride, "K", dev),
        _pool(V, f.pool, f.v_stride, "V", dev), _packed(page_table, _I32, f.table, "page_table", dev),
        _packed(q_begin, _I32, f.begin, "q_begin", dev), _packed(seq_lens, _I32, f.seq, "seq_lens", dev),
        window, n_sinks, sm_scale, _packed(O, f.out, (n, Hq, d), "O", dev),
        None if lse is None else _packed(lse, _F32, (n, Hq), "lse", dev), w, nw, _stream(stream, dev))
    if code:
        _check("jssa_paged_attn", code)


def pages_fork(L, src, dst, page_table, ref_count, seq_lens, ws, stream=None):
    """Sequence dst[i] (empty) becomes a copy of sequence src[i] that shares its pages."""
    dev, f = _device(), _facts(L)
    s, n = _list(src, "src", dev)
    code = load().jssa_pages_fork(
        C.byref(L), s, _packed(dst, _I32, (n,), "dst", dev), n,
        *_book(f, page_table, ref_count, seq_lens, dev), *_ws(ws, dev), _stream(stream, dev))
    if code:
        _check("jssa_pages_fork", code)


def pages_reserve(L, n_new, page_table, ref_count, seq_lens, copy_src, copy_dst, ws, stream=None):
    """Room for n_new[b] more tokens of every sequence, added to seq_lens; copy_src/copy_dst [B]
    name the shared pages to copy (pages_copy) before the append."""
    dev, f = _device(), _facts(L)
    code = load().jssa_pages_reserve(
        C.byref(L), _packed(n_new, _I32, f.seq, "n_new", dev), *_book(f, page_table, ref_count, seq_lens, dev),
        _packed(copy_src, _I32, f.seq, "copy_src", dev), _packed(copy_dst, _I32, f.seq, "copy_dst", dev),
        *_ws(ws, dev), _stream(stream, dev))
    if code:
        _check("jssa_pages_reserve", code)


def pages_release(L, ended, window: int, n_sinks: int, page_table, ref_count, seq_lens, ws, stream=None):
    """Give up all pages of the sequences with ended[b] != 0 and, with window > 0, the others' pages
    behind their last `window` tokens that hold none of the first n_sinks."""
    dev, f = _device(), _facts(L)
    _fits(window, n_sinks)
    code = load().jssa_pages_release(
        C.byref(L), None if ended is None else _packed(ended, _I32, f.seq, "ended", dev), window, n_sinks,
        *_book(f, page_table, ref_count, seq_lens, dev), *_ws(ws, dev), _stream(stream, dev))
    if code:
        _check("jssa_pages_release", code)


def pages_compact(L, page_table, ref_count, src, dst, n_moves, ws, stream=None):
    """Move the pages in use to the front of the pool (at most len(src) of them): the table and the
    counts now, the rows with pages_copy(..., src, dst, n_moves)."""
    dev, f = _device(), _facts(L)
    s, n = _list(src, "src", dev)
    code = load().jssa_pages_compact(
        C.byref(L), _packed(page_table, _I32, f.table, "page_table", dev),
        _packed(ref_count, _I32, f.ref, "ref_count", dev), s, _packed(dst, _I32, (n,), "dst", dev), n,
        _packed(n_moves, _I32, (1,), "n_moves", dev), *_ws(ws, dev), _stream(stream, dev))
    if code:
        _check("jssa_pages_compact", code)


def pages_copy(L, K, V, src, dst, count=None, ws=None, stream=None):
    """Copy page src[i] over page dst[i] in both pools, for every entry or the first count[0];
    negative entries are skipped."""
    dev, f = _device(), _facts(L)
    s, n = _list(src, "src", dev)
    code = load().jssa_pages_copy(
        C.byref(L), _pool(K, f.pool, f.k_stride, "K", dev), _pool(V, f.pool, f.v_stride, "V", dev), s,
        _packed(dst, _I32, (n,), "dst", dev), n,
        None if count is None else _packed(count, _I32, (1,), "count", dev), *_ws(ws, dev),
        _stream(stream, dev))
    if code:
        _check("jssa_pages_copy", code)
