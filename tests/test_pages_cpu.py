"""mla_page_resize and mla_page_fork without a GPU: refusals, and the oracle by hand."""
import ctypes

import numpy as np
import pytest

import oracle
import paged_mla_decode_09_gb300 as mla
from paged_mla_decode_09_gb300.build import build_library


@pytest.fixture(scope="module")
def lib():
    build_library()
    return mla.load_library()


def ptrs(n):
    return [ctypes.c_void_p((k + 1) << 24) for k in range(n)]


def _resize(lib, a=None, ws=1 << 40, **kw):
    d = dict(batch=2, num_pages=16, max_pages_per_req=5, table_stride=5, out_stride=5)
    d.update(kw)
    return lib.mla_page_resize(ctypes.byref(mla.MlaPageResizeDims(**d)), *(a or ptrs(6)), ws, None)


def _fork(lib, a=None, ws=1 << 40, **kw):
    d = dict(sources=2, children=3, num_layers=1, num_pages=16, max_pages_per_req=5, table_stride=5, out_stride=5,
             kv_dtype=0, layer_stride=0)
    d.update(kw)
    return lib.mla_page_fork(ctypes.byref(mla.MlaPageForkDims(**d)), *(a or ptrs(8)), ws, None)


def test_resize_refusals(lib):
    for bad in (dict(batch=0), dict(num_pages=0), dict(max_pages_per_req=0), dict(table_stride=4), dict(out_stride=4)):
        assert _resize(lib, **bad) == -1, bad
    big = dict(max_pages_per_req=1 << 25, table_stride=1 << 25, out_stride=1 << 25)
    for bad in (big, dict(num_pages=(1 << 30) + 1),
                dict(batch=1 << 16, max_pages_per_req=1 << 16, table_stride=1 << 16, out_stride=1 << 16)):
        assert _resize(lib, **bad) == -2, bad
    for k in range(6):
        a = ptrs(6)
        a[k] = None
        assert _resize(lib, a) == -1, k
        a = ptrs(6)
        a[k] = ctypes.c_void_p(a[k].value + (128 if k == 5 else 2))
        assert _resize(lib, a) == -3, k
    # outputs that overlap an input without being it
    for i, j in ((3, 1), (4, 2)):
        a = ptrs(6)
        a[i] = ctypes.c_void_p(a[j].value + 4)
        assert _resize(lib, a) == -1
    a = ptrs(6)
    a[3] = a[1]  # in place, but with another stride
    assert _resize(lib, a, out_stride=6) == -1
    assert _resize(lib, ws=256) == -4
    assert lib.mla_page_resize(None, *ptrs(6), 1 << 40, None) == -1
    for args in ((0, 5, 16), (2, 0, 16), (2, 5, 0), (2, 1 << 25, 16), (1 << 16, 1 << 16, 16)):
        assert lib.mla_page_resize_workspace_size(*args) == 0
    # no more ids are listed than there are pages, or entries
    assert lib.mla_page_resize_workspace_size(2, 5, 16) == lib.mla_page_resize_workspace_size(2, 5, 1 << 20)
    assert lib.mla_page_resize_workspace_size(200, 500, 100) == lib.mla_page_resize_workspace_size(200, 5000, 100)


def test_resize_refuses_overlaps(lib):
    """Each output and the workspace over each other buffer, from its first and
    over its last element; a vector in the gaps of a table's rows is none."""
    words = [2, 2 * 5, 16, 2 * 5, 16, 4 * 64]  # new_lens, table, counts, table_out, counts_out, workspace (256 B pieces)
    assert lib.mla_page_resize_workspace_size(2, 5, 16) == 768
    for out in (3, 4, 5):
        for other in range(6):
            if other == out or (out, other) in ((3, 1), (4, 2)):  # (in place)
                continue
            a = ptrs(6)
            a[out] = a[other]
            assert _resize(lib, a) == -1, (out, other)
            if other != 5 and out != 5:
                a[out] = ctypes.c_void_p(a[other].value + 4 * words[other] - 4)
                assert _resize(lib, a) == -1, (out, other)
                a[out] = ctypes.c_void_p(a[other].value + 4 * words[other])  # right behind it
                assert _resize(lib, a, ws=256) == -4, (out, other)
    a = ptrs(6)
    a[5] = ctypes.c_void_p(a[1].value - 512)  # its third piece reaches into the table
    assert _resize(lib, a) == -1
    # rows of 5 entries, 9 apart: lengths in the gap, at its end, and one further
    for at, rc in ((4, -1), (5, -4), (7, -4), (8, -1), (9, -1), (14, -4)):
        a = ptrs(6)
        a[0] = ctypes.c_void_p(a[3].value + 4 * at)
        assert _resize(lib, a, ws=256, out_stride=9) == rc, at


def test_fork_refusals(lib):
    for bad in (dict(sources=0), dict(children=0), dict(num_layers=0), dict(num_pages=0), dict(max_pages_per_req=0),
                dict(table_stride=4), dict(out_stride=4), dict(num_layers=2, layer_stride=16 * 64 * 1152 - 16)):
        assert _fork(lib, **bad) == -1, bad
    for bad in (dict(kv_dtype=2), dict(num_layers=65536, layer_stride=1 << 40), dict(num_pages=1 << 25),
                dict(max_pages_per_req=1 << 25, table_stride=1 << 25, out_stride=1 << 25)):
        assert _fork(lib, **bad) == -2, bad
    assert _fork(lib, num_layers=2, layer_stride=16 * 64 * 1152 + 8) == -3
    for k in range(8):
        a = ptrs(8)
        a[k] = None
        assert _fork(lib, a) == -1, k
        a = ptrs(8)
        a[k] = ctypes.c_void_p(a[k].value + (128 if k == 7 else 8 if k == 4 else 2))
        assert _fork(lib, a) == -3, k
    for at in (0, 4, 9 * 4):  # the tables share an element: 2 rows of 5 entries
        a = ptrs(8)
        a[5] = ctypes.c_void_p(a[2].value + at)
        assert _fork(lib, a) == -1, at
    a = ptrs(8)
    a[6] = ctypes.c_void_p(a[3].value + 4)
    assert _fork(lib, a) == -1
    assert _fork(lib, ws=256) == -4
    assert lib.mla_page_fork(None, *ptrs(8), 1 << 40, None) == -1
    assert lib.mla_page_fork_workspace_size(2, 0, 5, 16) == 0


def test_fork_refuses_overlaps(lib):
    """As for resize; 2 sources, 3 children, 5 columns, 16 pages."""
    words = {0: 3, 1: 2, 2: 10, 3: 16, 5: 15, 6: 16, 7: 256}
    assert lib.mla_page_fork_workspace_size(2, 3, 5, 16) == 1024
    for out in (5, 6, 7):
        for other in words:
            if other == out or (out, other) == (6, 3):  # (in place)
                continue
            a = ptrs(8)
            a[out] = a[other]
            assert _fork(lib, a) == -1, (out, other)
            if out == 7:
                a[7] = ctypes.c_void_p(a[other].value - 768)  # its fourth piece reaches into the other
                assert _fork(lib, a) == -1, other
                continue
            a[out] = ctypes.c_void_p(a[other].value + 4 * words[other] - 4)
            assert _fork(lib, a) == -1, (out, other)
            a[out] = ctypes.c_void_p(a[other].value + 4 * words[other])  # right behind it
            assert _fork(lib, a, ws=256) == -4, (out, other)
    # rows of 5 entries, 9 apart: sources in the gap, at its end, and one further
    for at, rc in ((4, -1), (5, -4), (6, -4), (7, -1), (9, -1), (23, -4)):
        a = ptrs(8)
        a[0] = ctypes.c_void_p(a[5].value + 4 * at)
        assert _fork(lib, a, ws=256, out_stride=9) == rc, at


def test_binding_refuses_what_the_library_cannot_see(lib):
    torch = pytest.importorskip("torch")
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.mla_page_resize(z, z, z, z, z, z)
    with pytest.raises(ValueError):
        mla.mla_page_fork(z, z, z, z, z, z, z, z)
    table = torch.zeros(3, 4, dtype=torch.int32)
    mla._check_table("t", table, 3)
    mla._check_table("t", torch.zeros(3, 9, dtype=torch.int32)[:, 2:6], 3)
    for bad in (table.long(), table.t(), table[:2], table[:1].expand(3, 4), table[0]):
        with pytest.raises(ValueError):
            mla._check_table("t", bad, 3)


def test_resize_ref_by_hand():
    table = np.array([[3, 1, -1], [3, 0, 2], [-1, -1, -1]], np.int32)
    refs = np.array([1, 1, 1, 2, 0, 0], np.int32)
    t, r, status = oracle.page_resize_ref([129, 0, 64], table, refs)
    assert t.tolist() == [[3, 1, 0], [-1, -1, -1], [2, -1, -1]] and r.tolist() == [1, 1, 1, 1, 0, 0] and status == 0
    t, r, status = oracle.page_resize_ref([192, 192, 192], table, refs)
    assert t.tolist() == [[3, 1, 4], [3, 0, 2], [5, -1, -1]] and status == 512


def test_fork_ref_by_hand():
    table = np.array([[3, 1, -1], [2, -1, -1]], np.int32)
    refs = np.array([0, 1, 1, 1, 0], np.int32)
    cache = np.arange(5 * 64).reshape(1, 5, 64, 1).repeat(576, axis=3)
    t, r, c, status = oracle.page_fork_ref([0, -1, 0, 1], [66, 64], table, refs, cache)
    assert t.tolist() == [[3, 0, -1], [-1] * 3, [3, 4, -1], [2, -1, -1]] and r.tolist() == [1, 1, 2, 3, 1] and status == 0
    assert c[0, 0, :3, 0].tolist() == [64, 65, 2] and c[0, 4, :3, 0].tolist() == [64, 65, 4 * 64 + 2]
