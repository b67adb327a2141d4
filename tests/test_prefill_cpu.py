"""mla_prefill and mla_decode_window without a GPU: refusals of the C entry
points and the binding, and the pins of the oracle that the GPU tests use."""
import ctypes

import numpy as np
import pytest

import chunk_cases as K
import oracle
import paged_mla_decode_09_gb300 as mla
from paged_mla_decode_09_gb300.build import build_library


@pytest.fixture(scope="module")
def lib():
    build_library()
    return mla.load_library()


P = ctypes.c_void_p(256)


def _dims(**kw):
    d = dict(batch=2, num_heads=16, total_q=10, page_size=64, num_pages=16, max_pages_per_req=5, page_table_stride=5,
             kv_dtype=0)
    d.update(kw)
    return mla.MlaPrefillDims(**d)


def _wdims(**kw):
    d = dict(batch=2, num_heads=16, q_len=1, page_size=64, num_pages=16, max_pages_per_req=5, page_table_stride=5,
             kv_dtype=0)
    d.update(kw)
    return mla.MlaDims(**d)


def _prefill(lib, d, ptrs=None, window=0, sinks=0, scale=1.0, kv_scale=1.0):
    a = [P] * 9 if ptrs is None else ptrs
    return lib.mla_prefill(ctypes.byref(d), *a[:6], window, sinks, scale, kv_scale, *a[6:], 1 << 40, None)


def _window(lib, d, ptrs=None, window=8, sinks=0, scale=1.0, kv_scale=1.0):
    a = [P] * 8 if ptrs is None else ptrs
    return lib.mla_decode_window(ctypes.byref(d), *a[:5], window, sinks, scale, kv_scale, *a[5:], 1 << 40, None)


@pytest.mark.parametrize("bad", [dict(batch=0), dict(num_heads=0), dict(total_q=0), dict(num_pages=0),
                                 dict(max_pages_per_req=0), dict(page_table_stride=4)])
def test_prefill_refuses_bad_dims(lib, bad):
    assert _prefill(lib, _dims(**bad)) == -1
    assert lib.mla_prefill_workspace_size(ctypes.byref(_dims(**bad)), 0) == 0


@pytest.mark.parametrize("bad", [dict(page_size=32), dict(kv_dtype=2), dict(total_q=1 << 28),
                                 dict(max_pages_per_req=1 << 26, page_table_stride=1 << 26), dict(num_pages=1 << 26),
                                 dict(batch=(1 << 30) + 1, max_pages_per_req=1, page_table_stride=1),
                                 dict(total_q=1 << 20, num_heads=128, max_pages_per_req=1 << 12,
                                      page_table_stride=1 << 12)])
def test_prefill_refuses_what_it_does_not_support(lib, bad):
    assert _prefill(lib, _dims(**bad)) == -2
    assert lib.mla_prefill_workspace_size(ctypes.byref(_dims(**bad)), 0) == 0


def test_prefill_refuses_bad_arguments(lib):
    d = _dims()
    for k in range(9):
        ptrs = [P] * 9
        ptrs[k] = None
        assert _prefill(lib, d, ptrs) == -1, k
    for k, off in ((0, 16), (1, 16), (2, 8), (3, 2), (4, 2), (5, 2), (6, 16), (7, 2), (8, 128)):
        ptrs = [P] * 9
        ptrs[k] = ctypes.c_void_p(256 + off)
        assert _prefill(lib, d, ptrs) == -3, k
    assert _prefill(lib, d, window=-1) == -1
    assert _prefill(lib, d, sinks=-1) == -1
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _prefill(lib, d, scale=s) == -1
        assert _prefill(lib, _dims(kv_dtype=1), kv_scale=s) == -1
    assert lib.mla_prefill(None, *[P] * 6, 0, 0, 1.0, 1.0, P, P, P, 1 << 40, None) == -1


def test_decode_window_refuses_bad_arguments(lib):
    assert _window(lib, _wdims(), window=0) == -1
    assert _window(lib, _wdims(), window=-3) == -1
    assert _window(lib, _wdims(), sinks=-1) == -1
    assert _window(lib, _wdims(q_len=0)) == -1
    assert _window(lib, _wdims(batch=0)) == -1
    assert _window(lib, _wdims(page_size=16)) == -2
    assert _window(lib, _wdims(batch=1 << 16, q_len=1 << 10, num_heads=128)) == -2
    for k in range(8):
        ptrs = [P] * 8
        ptrs[k] = None
        assert _window(lib, _wdims(), ptrs) == -1, k
    assert lib.mla_decode_window_workspace_size(ctypes.byref(_wdims(batch=0)), 0) == 0


def _tensors():
    torch = pytest.importorskip("torch")
    c = K.make([3, 2], [70, 100], heads=4, seed=1)
    bf = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16)  # noqa: E731
    T = c.q_nope.shape[0]
    t = dict(q_nope=bf(c.q_nope), q_pe=bf(c.q_pe), kv_cache=bf(c.kv_cache), page_table=torch.from_numpy(c.page_table),
             seq_lens=torch.from_numpy(c.seq_lens), cu_q_lens=torch.from_numpy(c.cu),
             out=torch.empty(T, 4, 512, dtype=torch.bfloat16), lse=torch.empty(T, 4),
             workspace=torch.empty(4096, dtype=torch.uint8))
    return torch, t


def test_binding_layout_checks():
    torch, t = _tensors()
    mla._check_prefill_tensors(**t)
    bad = [("q_nope", t["q_nope"][None]), ("q_nope", t["q_nope"].float()), ("q_nope", t["q_nope"][:1].expand(5, 4, 512)),
           ("q_pe", t["q_pe"][:4]), ("out", t["out"].float()), ("lse", t["lse"].t().contiguous().t()),
           ("cu_q_lens", t["cu_q_lens"][:2]), ("cu_q_lens", t["cu_q_lens"].long()), ("seq_lens", t["seq_lens"][:, None]),
           ("page_table", t["page_table"][:1]), ("kv_cache", t["kv_cache"][..., :512]),
           ("workspace", torch.empty(64, 2, dtype=torch.uint8).t())]
    for name, x in bad:
        with pytest.raises((ValueError, TypeError)):
            mla._check_prefill_tensors(**{**t, name: x})
    with pytest.raises(ValueError):
        mla.mla_prefill(*[t[k] for k in ("q_nope", "q_pe", "kv_cache", "page_table", "seq_lens", "cu_q_lens")], 0, 0,
                        1.0, 1.0, t["out"], t["lse"], t["workspace"])  # CPU tensors
    for v in (-1, 1 << 31):
        with pytest.raises(ValueError):
            mla._int32_arg("window", v)


# ---- the oracle ----

def test_seen_keys_by_hand():
    assert oracle.seen_keys(5, 0, 3).tolist() == [0, 1, 2, 3, 4, 5]
    assert oracle.seen_keys(5, 2, 0).tolist() == [4, 5]
    assert oracle.seen_keys(5, 2, 3).tolist() == [0, 1, 2, 4, 5]
    assert oracle.seen_keys(5, 1, 1).tolist() == [0, 5]
    assert oracle.seen_keys(5, 2, 5).tolist() == [0, 1, 2, 3, 4, 5]
    assert oracle.seen_keys(0, 9, 9).tolist() == [0]


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_oracle_without_a_window_is_the_decode(kv_dtype):
    c = K.make([2, 2], [70, 130], heads=4, kv_dtype=kv_dtype, seed=2)
    out, lse = oracle.mla_prefill_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, 0, 5, c.scale,
                                      c.kv_scale, kv_dtype)
    ro, rl = oracle.mla_decode_ref(c.q_nope.reshape(2, 2, 4, 512), c.q_pe.reshape(2, 2, 4, 64), c.kv_cache,
                                   c.page_table, c.seq_lens, 2, c.scale, c.kv_scale, kv_dtype)
    assert np.allclose(out, ro.reshape(4, 4, 512), rtol=0, atol=1e-12)
    assert np.allclose(lse, rl.reshape(4, 4), rtol=0, atol=1e-12)


def test_oracle_window_equals_a_mask_over_all_scores():
    c = K.make([4], [200], heads=3, seed=4)  # every page present; the mask is applied to full score rows
    window, sinks = 37, 66
    out, lse = oracle.mla_prefill_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, window, sinks, 0.1)
    k = oracle.bf16_bits_to_f64(c.kv_cache[c.page_table[0]].reshape(-1, 576)[:200])
    for i in range(4):
        p = 196 + i
        q = np.concatenate([oracle.bf16_bits_to_f64(c.q_nope[i]), oracle.bf16_bits_to_f64(c.q_pe[i])], axis=1)
        s = q @ k.T * 0.1
        t = np.arange(200)
        s[:, ~((t <= p) & ((p - t < window) | (t < sinks)))] = -np.inf
        w = np.exp(s)
        assert np.allclose(lse[i], np.log(w.sum(axis=1)), atol=1e-12)
        assert np.allclose(out[i], (w / w.sum(axis=1, keepdims=True)) @ k[:, :512], atol=1e-12)


def test_oracle_full_window_is_no_window():
    c = K.make([3, 1], [90, 65], heads=2, seed=6)
    a = oracle.mla_prefill_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, 0, 0, 0.1)
    b = oracle.mla_prefill_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, 90, 0, 0.1)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
