"""mla_rope_pack without a GPU: frequencies and plans (host code), refusals,
and the oracle's pins."""
import ctypes
import math

import numpy as np
import pytest

import oracle
import paged_mla_decode_09_gb300 as mla
from paged_mla_decode_09_gb300.build import build_library


@pytest.fixture(scope="module")
def lib():
    build_library()
    return mla.load_library()


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(factor=4.0), dict(factor=40.0, original_len=4096),
                                dict(factor=8.0, original_len=8192, fast=4.0, slow=0.5, base=1e6)])
@pytest.mark.parametrize("dim", [16, 32, 48, 64])
def test_frequencies(lib, dim, kw):
    got = mla.mla_rope_frequencies(dim, **kw)
    want = oracle.rope_frequencies_ref(dim, **{"base": 10000.0, **kw})
    assert len(got) == dim // 2
    assert np.allclose(got, want, rtol=1e-14, atol=0)  # pow and a few 64-bit operations
    assert got[0] == 1.0 if kw.get("factor", 1.0) == 1.0 or kw.get("original_len") else got[0] == 1.0 / kw["factor"]


def test_frequencies_by_index_by_hand(lib):
    """R = 64, base 10000, 4096 positions: index 10.5 turns 32 times and 22.5
    once, so pairs up to 10 stay, pairs from 23 on are divided by 40."""
    assert 10 < 32 * math.log(4096 / (2 * math.pi * 32)) / math.log(10000) < 11
    assert 22 < 32 * math.log(4096 / (2 * math.pi)) / math.log(10000) < 23
    f = [10000.0 ** (-i / 32) for i in range(32)]
    got = mla.mla_rope_frequencies(64, factor=40.0, original_len=4096, ramp="index")
    assert np.allclose(got[:11], f[:11], rtol=1e-14, atol=0) and np.allclose(got[23:], np.asarray(f[23:]) / 40, rtol=1e-14, atol=0)
    for i in range(11, 23):
        assert abs(got[i] / f[i] - ((23 - i) + (i - 10) / 40) / 13) < 1e-14
    assert abs(got[16] / f[16] - 0.55) < 1e-14
    # the ramp over turns is another one in just these twelve pairs
    turns = mla.mla_rope_frequencies(64, factor=40.0, original_len=4096)
    assert turns == mla.mla_rope_frequencies(64, factor=40.0, original_len=4096, ramp="turns")
    assert [i for i in range(32) if abs(turns[i] / got[i] - 1) > 1e-12] == list(range(11, 23))
    # without a length, or a factor, there is no ramp
    assert mla.mla_rope_frequencies(64, factor=40.0, ramp="index") == mla.mla_rope_frequencies(64, factor=40.0)
    assert mla.mla_rope_frequencies(64, original_len=4096, ramp="index") == mla.mla_rope_frequencies(64)
    plan = mla.mla_rope_plan(64, factor=40.0, original_len=4096, ramp="index")
    assert list(plan.turn) == list(mla.mla_rope_plan(64, frequencies=got).turn)


@pytest.mark.parametrize("kw", [dict(factor=40.0, original_len=4096), dict(factor=4.0, original_len=32768, base=1e6),
                                dict(factor=8.0, original_len=8192, fast=4.0, slow=0.5, base=1e6),
                                dict(factor=2.0, original_len=3), dict(factor=2.0, original_len=2**31 - 1),
                                dict(factor=2.0, original_len=2**31 - 1, base=2.0),
                                dict(factor=3.0, original_len=1000, fast=1.01, slow=1.0)])
@pytest.mark.parametrize("dim", [16, 32, 48, 64])
def test_frequencies_by_index(lib, dim, kw):
    got = mla.mla_rope_frequencies(dim, ramp="index", **kw)
    assert np.allclose(got, oracle.rope_frequencies_by_index_ref(dim, **{"base": 10000.0, **kw}), rtol=1e-13, atol=0)
    assert all(a >= b for a, b in zip(got, got[1:]))  # never faster than the pair before


def test_frequencies_by_index_refusals(lib):
    for kw in (dict(base=0.5), dict(base=float("nan")), dict(factor=0.9), dict(original_len=-1),
               dict(original_len=10, fast=1.0, slow=1.0), dict(original_len=10, fast=float("nan")),
               dict(original_len=10, slow=0.0), dict(original_len=10, slow=-1.0), dict(original_len=10, base=1.0)):
        with pytest.raises((mla.MlaError, ValueError)):
            mla.mla_rope_frequencies(64, **{"factor": 2.0, **kw}, ramp="index")
    with pytest.raises(mla.MlaError):
        mla.mla_rope_frequencies(40, ramp="index")
    for ramp in ("linear", None, 1, []):
        with pytest.raises(ValueError):
            mla.mla_rope_frequencies(64, ramp=ramp)
        with pytest.raises(ValueError):
            mla.mla_rope_plan(64, ramp=ramp)
    assert lib.mla_rope_frequencies_by_index(16, 10.0, 1.0, 0, 1.0, 1.0, None) == -1


def test_plan_holds_turns(lib):
    plan = mla.mla_rope_plan(32, interleaved=False, amplitude=1.25)
    assert plan.rotary_dim == 32 and plan.interleaved == 0 and plan.amplitude == 1.25
    for f, t in zip(mla.mla_rope_frequencies(32), plan.turn):
        assert abs(t / 2**64 - f / (2 * math.pi)) <= 2.0**-52 * f
    assert list(plan.turn)[16:] == [0] * 16
    plan = mla.mla_rope_plan(16, frequencies=[0.0, 6.28] + [0.5] * 6)
    assert plan.turn[0] == 0


def test_frequency_and_plan_refusals(lib):
    for kw in (dict(base=0.5), dict(base=float("nan")), dict(base=float("inf")), dict(factor=0.9),
               dict(factor=float("inf")), dict(original_len=-1), dict(factor=2.0, original_len=10, fast=1.0, slow=1.0),
               dict(factor=2.0, original_len=10, fast=float("nan"))):
        with pytest.raises((mla.MlaError, ValueError)):
            mla.mla_rope_frequencies(64, **kw)
    for dim in (0, 8, 40, 80, 2):
        with pytest.raises(mla.MlaError):
            mla.mla_rope_frequencies(dim)
        with pytest.raises(mla.MlaError):
            mla.mla_rope_plan(dim, frequencies=[0.1] * (dim // 2))
    for f in (-0.1, 6.2831854, float("nan"), float("inf")):
        with pytest.raises(mla.MlaError):
            mla.mla_rope_plan(16, frequencies=[f] * 8)
    for a in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(mla.MlaError):
            mla.mla_rope_plan(16, amplitude=a)
    with pytest.raises(ValueError):
        mla.mla_rope_plan(16, frequencies=[0.1] * 7)
    assert lib.mla_rope_frequencies(16, 10.0, 1.0, 0, 1.0, 1.0, None) == -1
    assert lib.mla_rope_plan_init(16, 1, 1.0, None, ctypes.byref(mla.MlaRopePlan())) == -1


def _pack(lib, ptrs=None, kv_scale=1.0, plan=None, **kw):
    d = dict(batch=2, num_heads=16, total_q=6, num_pages=16, max_pages_per_req=5, page_table_stride=5, kv_dtype=0,
             reserved=0, q_token_stride=1024, q_head_stride=64, row_stride=576)
    d.update(kw)
    a = [ctypes.c_void_p((k + 1) << 24) for k in range(9)] if ptrs is None else ptrs
    plan = mla.mla_rope_plan(64) if plan is None else plan
    return lib.mla_rope_pack(ctypes.byref(mla.MlaRopeDims(**d)), ctypes.byref(plan), *a[:6], kv_scale, *a[6:], None)


def test_pack_refusals(lib):
    for bad in (dict(batch=0), dict(num_heads=0), dict(total_q=0), dict(num_pages=0), dict(max_pages_per_req=0),
                dict(page_table_stride=4), dict(q_token_stride=56), dict(q_head_stride=56), dict(row_stride=568)):
        assert _pack(lib, **bad) == -1, bad
    for bad in (dict(kv_dtype=2), dict(num_heads=65537), dict(total_q=1 << 28), dict(row_stride=1 << 41),
                dict(max_pages_per_req=1 << 26, page_table_stride=1 << 26)):
        assert _pack(lib, **bad) == -2, bad
    for bad in (dict(q_token_stride=1028), dict(q_head_stride=68), dict(row_stride=580)):
        assert _pack(lib, **bad) == -3, bad
    good = [ctypes.c_void_p((k + 1) << 24) for k in range(9)]
    for k in range(9):
        off = ctypes.c_void_p(good[k].value + (8 if k in (0, 1, 6, 7) else 2))
        assert _pack(lib, good[:k] + [off] + good[k + 1:]) == -3, k
        if k != 2:  # no positions: slots
            assert _pack(lib, good[:k] + [None] + good[k + 1:]) == -1, k
    for s in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert _pack(lib, kv_dtype=1, kv_scale=s) == -1
    # outputs over a part of the input, or over the input with gaps
    assert _pack(lib, good[:6] + [ctypes.c_void_p(good[0].value + 128)] + good[7:]) == -1
    assert _pack(lib, good[:6] + [good[0]] + good[7:], q_token_stride=2048) == -1
    plan = mla.mla_rope_plan(64)
    plan.rotary_dim = 24
    assert _pack(lib, plan=plan) == -2
    plan = mla.mla_rope_plan(64)
    plan.amplitude = float("nan")
    assert _pack(lib, plan=plan) == -1


def test_pack_refuses_outputs_over_inputs(lib):
    """The rotated queries and the status word over what blocks read while others
    write; 6 tokens, 16 heads, 2 requests, 5 pages.  (q_pe is off its alignment,
    which is looked at next: no call gets further.)"""
    good = [ctypes.c_void_p((k + 1) << 24) for k in range(9)]
    good[0] = ctypes.c_void_p((1 << 24) + 8)
    assert _pack(lib, good) == -3
    words = {1: 6 * 288, 2: 6, 3: 2 * 5, 4: 2, 5: 3, 6: 6 * 16 * 32, 8: 1}
    for out in (6, 8):
        for other in words:
            if other != out:
                for at in (0, words[other] - 1):
                    a = list(good)
                    a[out] = ctypes.c_void_p(a[other].value + 4 * at)
                    assert _pack(lib, a) == -1, (out, other, at)
                a[out] = ctypes.c_void_p(a[other].value + 4 * words[other])  # right behind it
                assert _pack(lib, a) == -3, (out, other)
    # a status word between the rows, and between the table's
    for k, wide, n in ((1, dict(row_stride=584), 288), (3, dict(page_table_stride=9), 5)):
        for at, rc in ((n - 1, -1), (n, -3), (n + 3, -3), (n + 4, -1)):
            a = list(good)
            a[8] = ctypes.c_void_p(a[k].value + 4 * at)
            assert _pack(lib, a, **wide) == rc, (k, at)
    # without positions there is nothing to overlap
    a = list(good)
    a[2] = None
    assert _pack(lib, a) == -3


def test_binding_refuses_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    z = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.mla_rope_pack(mla.mla_rope_plan(64), z, z, None, z, z, z, 1.0, z, z, z)


def test_rotation_keeps_lengths_and_differences():
    """A rotation keeps a pair's length, and the product of two rotated vectors
    depends on the difference of their positions alone."""
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((1, 64)), rng.standard_normal((1, 64))
    f = oracle.rope_frequencies_ref(64, 10000.0)
    for inter in (True, False):
        a, b = oracle.rotate_ref(x, [1000], f, inter), oracle.rotate_ref(y, [990], f, inter)
        assert np.isclose(np.linalg.norm(a), np.linalg.norm(x))
        c, d = oracle.rotate_ref(x, [10], f, inter), oracle.rotate_ref(y, [0], f, inter)
        assert np.isclose((a * b).sum(), (c * d).sum())
        assert np.array_equal(d, y)
    # pairs: neighbours, or half the rotated part apart; the rest passes
    one = np.zeros((1, 64))
    one[0, 2] = 1.0
    assert np.flatnonzero(oracle.rotate_ref(one, [1], f[:8], True)).tolist() == [2, 3]
    assert np.flatnonzero(oracle.rotate_ref(one, [1], f[:8], False)).tolist() == [2, 10]
