"""The paged-cache entry points on the CPU: what the library and the binding refuse before any
CUDA call."""
import ctypes as C
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 256-byte aligned and non-null; validation answers before it is used


@pytest.fixture(scope="module")
def lib():
    from token_level_sparse_jssa_b200 import build
    build.build()
    from token_level_sparse_jssa_b200 import _binding
    return _binding.load()


def _layout(**kw):
    from token_level_sparse_jssa_b200 import PagedLayout
    L = PagedLayout()
    L.B, L.Hq, L.Hkv, L.d, L.page_size = kw.get("B", 3), kw.get("Hq", 8), kw.get("Hkv", 2), kw.get("d", 128), \
        kw.get("page", 16)
    L.n_pages, L.max_pages, L.out_dtype = kw.get("n_pages", 40), kw.get("max_pages", 9), kw.get("out", 0)
    for i, v in enumerate(kw.get("stride", (L.Hkv * L.page_size * L.d, L.page_size * L.d, L.d))):
        L.k_stride[i] = v
        L.v_stride[i] = v
    for i, v in enumerate(kw.get("v_stride", ())):
        L.v_stride[i] = v
    return L


def _append(lib, L, kn=FAKE, vn=FAKE, stride=256, n=5, k=FAKE, v=FAKE, table=FAKE, qb=FAKE, sl=FAKE, ws=FAKE,
            ws_bytes=1 << 40):
    return lib.jssa_paged_append_kv(C.byref(L) if L is not None else None, kn, vn, stride, n, k, v, table, qb, sl,
                                    C.c_void_p(ws), ws_bytes, None)


def _attn(lib, L, q=FAKE, stride=1024, n=5, max_q=2, k=FAKE, v=FAKE, table=FAKE, qb=FAKE, sl=FAKE, window=0, sinks=0,
          scale=0.1, o=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40):
    return lib.jssa_paged_attn(C.byref(L) if L is not None else None, q, stride, n, max_q, k, v, table, qb, sl, window,
                               sinks, C.c_float(scale), o, lse, C.c_void_p(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(Hq=7), 1), (dict(Hkv=0), 1), (dict(out=2), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1),
    (dict(page=0), 1), (dict(d=0), 1),
    (dict(stride=(4096, 2048, 132)), 1),     # strides of whole 16-byte words
    (dict(stride=(4096, 2048, 64)), 1),      # rows that overlap
    (dict(v_stride=(-8, 2048, 128)), 1),
    (dict(stride=(1 << 39, 2048, 128)), 1),
    (dict(d=96), 2), (dict(d=576), 2), (dict(B=1025), 2), (dict(Hq=129, Hkv=1), 2), (dict(page=24), 2),
    (dict(page=8), 2), (dict(max_pages=1 << 28), 2),
])
def test_bad_layouts(lib, kw, code):
    L = _layout(**kw)
    n = C.c_size_t(0)
    ws = (C.c_void_p(FAKE), 1 << 40, None)
    assert lib.jssa_paged_workspace_size(C.byref(L), 1, C.byref(n)) == code
    assert _append(lib, L) == code
    assert _attn(lib, L) == code
    assert lib.jssa_pages_fork(C.byref(L), FAKE, FAKE, 2, FAKE, FAKE, FAKE, *ws) == code
    assert lib.jssa_pages_reserve(C.byref(L), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, *ws) == code
    assert lib.jssa_pages_release(C.byref(L), FAKE, 0, 0, FAKE, FAKE, FAKE, *ws) == code
    assert lib.jssa_pages_compact(C.byref(L), FAKE, FAKE, FAKE, FAKE, 2, FAKE, *ws) == code
    assert lib.jssa_pages_copy(C.byref(L), FAKE, FAKE, FAKE, FAKE, 2, None, *ws) == code


def test_append_arguments(lib):
    L = _layout()
    assert _append(lib, None) == 1
    for kw in (dict(kn=None), dict(vn=None), dict(k=None), dict(v=None), dict(table=None), dict(qb=None), dict(sl=None),
               dict(kn=FAKE + 8), dict(v=FAKE + 2), dict(table=FAKE + 2), dict(stride=255), dict(stride=260),
               dict(stride=1 << 40), dict(n=-1), dict(n=1 << 31)):
        assert _append(lib, L, **kw) == 1, kw
    assert _append(lib, L, n=0, kn=None, vn=None, k=None, v=None, table=None, qb=None, sl=None, ws=None) == 0
    assert _append(lib, L, ws=None) == 3
    assert _append(lib, L, ws=FAKE + 16) == 3


def test_attention_arguments(lib):
    L = _layout()
    assert _attn(lib, None) == 1
    for kw in (dict(q=None), dict(o=None), dict(k=None), dict(v=None), dict(table=None), dict(qb=None), dict(sl=None),
               dict(q=FAKE + 8), dict(o=FAKE + 4), dict(lse=FAKE + 2), dict(stride=1023), dict(stride=1028),
               dict(stride=1 << 40), dict(n=-1), dict(n=1 << 31), dict(max_q=-1), dict(window=-1), dict(sinks=-1),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2.5e38)):
        assert _attn(lib, L, **kw) == 1, kw
    assert _attn(lib, L, n=0, q=None, o=None, ws=None) == 0
    assert _attn(lib, L, max_q=0, q=None, o=None, ws=None) == 0
    assert _attn(lib, L, ws=None) == 3
    assert _attn(lib, L, ws=FAKE + 64) == 3


def test_page_operation_arguments(lib):
    L = _layout()
    ws = (C.c_void_p(FAKE), 1 << 40, None)
    none = (None, 0, None)
    fork = [FAKE, FAKE, 2, FAKE, FAKE, FAKE]
    reserve = [FAKE] * 6
    release = [FAKE, 4, 1, FAKE, FAKE, FAKE]
    compact = [FAKE, FAKE, FAKE, FAKE, 2, FAKE]
    copy = [FAKE, FAKE, FAKE, FAKE, 2, FAKE]
    for fn, args, optional in ((lib.jssa_pages_fork, fork, ()), (lib.jssa_pages_reserve, reserve, ()),
                               (lib.jssa_pages_release, release, (0,)), (lib.jssa_pages_compact, compact, ()),
                               (lib.jssa_pages_copy, copy, (5,))):
        assert fn(C.byref(L), *args, *none) == 3
        assert fn(C.byref(L), *args, C.c_void_p(FAKE + 8), 1 << 40, None) == 3
        for i, a in enumerate(args):
            if a != FAKE:
                continue
            if i not in optional:
                assert fn(C.byref(L), *(args[:i] + [None] + args[i + 1:]), *ws) == 1
            assert fn(C.byref(L), *(args[:i] + [FAKE + 2] + args[i + 1:]), *ws) == 1
    for n in (-1, 65536):
        assert lib.jssa_pages_fork(C.byref(L), FAKE, FAKE, n, FAKE, FAKE, FAKE, *ws) == 1
    assert lib.jssa_pages_fork(C.byref(L), None, None, 0, None, None, None, *none) == 0
    assert lib.jssa_pages_release(C.byref(L), FAKE, -1, 0, FAKE, FAKE, FAKE, *ws) == 1
    assert lib.jssa_pages_release(C.byref(L), FAKE, 5, -1, FAKE, FAKE, FAKE, *ws) == 1
    assert lib.jssa_pages_compact(C.byref(L), FAKE, FAKE, FAKE, FAKE, 0, FAKE, *ws) == 1
    assert lib.jssa_pages_copy(C.byref(L), FAKE, FAKE, FAKE, FAKE, -1, None, *ws) == 1
    assert lib.jssa_pages_copy(C.byref(L), None, None, None, None, 0, None, *none) == 0


def test_workspace_size_arguments(lib):
    n = C.c_size_t(0)
    assert lib.jssa_paged_workspace_size(None, 1, C.byref(n)) == 1
    assert lib.jssa_paged_workspace_size(C.byref(_layout()), -1, C.byref(n)) == 1
    assert lib.jssa_paged_workspace_size(C.byref(_layout()), 1, None) == 1


def test_layout_struct_matches_header(tmp_path):
    from token_level_sparse_jssa_b200 import PagedLayout
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "jssa.h"\nint main(void){ printf("%zu %zu %d", '
                   'sizeof(jssa_paged_layout), offsetof(jssa_paged_layout, v_stride), JSSA_DEV_NO_PAGES); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    size, off, flag = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    from token_level_sparse_jssa_b200 import DEV_NO_PAGES
    assert (size, off, flag) == (C.sizeof(PagedLayout), PagedLayout.v_stride.offset, DEV_NO_PAGES)


def test_make_paged_layout():
    import token_level_sparse_jssa_b200 as jssa
    K = torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16).transpose(1, 2)
    V = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)
    L = jssa.make_paged_layout(K, V, torch.zeros(3, 4, dtype=torch.int32), 8, jssa.OUT_BF16)
    assert (L.B, L.Hq, L.Hkv, L.d, L.page_size, L.n_pages, L.max_pages, L.out_dtype) == (3, 8, 2, 64, 16, 6, 4, 1)
    assert list(L.k_stride) == [2048, 64, 128] and list(L.v_stride) == [2048, 1024, 64]
    with pytest.raises(ValueError):
        jssa.make_paged_layout(K, V[:5], torch.zeros(3, 4, dtype=torch.int32), 8)
    with pytest.raises(ValueError):
        jssa.make_paged_layout(K, V, torch.zeros(3, dtype=torch.int32), 8)


def test_host_tensors_are_refused():
    import token_level_sparse_jssa_b200 as jssa
    K, V = torch.zeros(2, 6, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(3, 4, dtype=torch.int32)
    L = jssa.make_paged_layout(K, V, table, 8)
    n = torch.zeros(3, dtype=torch.int32)
    ref = torch.zeros(6, dtype=torch.int32)
    rows = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: jssa.paged_append_kv(L, rows, rows, K, V, table, n, n, n),
                 lambda: jssa.paged_attn(L, rows, K, V, table, n, 1, n, 0, 0, 0.1, rows, None, n),
                 lambda: jssa.pages_fork(L, n, n, table, ref, n, n),
                 lambda: jssa.pages_reserve(L, n, table, ref, n, n, n, n),
                 lambda: jssa.pages_release(L, n, 0, 0, table, ref, n, n),
                 lambda: jssa.pages_compact(L, table, ref, n, n, n, n),
                 lambda: jssa.pages_copy(L, K, V, n, n, None, n)):
        with pytest.raises(ValueError):
            call()


def test_a_changed_layout_is_seen(monkeypatch):
    # what a call derives from a layout's fields follows the fields' present values
    import token_level_sparse_jssa_b200 as jssa
    from token_level_sparse_jssa_b200 import _paged
    monkeypatch.setattr(_paged, "_device", lambda: -1)      # where host tensors say they are
    K, V = torch.zeros(2, 6, 2, 16, 64, dtype=torch.bfloat16)
    L = jssa.make_paged_layout(K, V, torch.zeros(3, 4, dtype=torch.int32), 8)
    assert _paged._pool(K, _paged._facts(L).pool, _paged._facts(L).k_stride, "K", -1) == K.data_ptr()
    L.n_pages = 5
    L.k_stride[0] = 4096
    f = _paged._facts(L)
    assert f.pool == (5, 2, 16, 64) and f.k_stride == (4096, 1024, 64, 1)
    with pytest.raises(ValueError):
        _paged._pool(K, f.pool, f.k_stride, "K", -1)
    with pytest.raises(ValueError):
        _paged._pool(K[:5], f.pool, f.k_stride, "K", -1)
