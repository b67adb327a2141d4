"""scale * kv_scale * log2(e) is one fp32 factor of every score of mla_prefill,
mla_decode_window and mla_attn_mass: the entry points refuse one that is 0 or
not finite, where each factor alone is fine.  (The calls that are let through
come with a workspace too small to launch anything.)"""
import ctypes

import pytest

import paged_mla_decode_09_gb300 as mla
from paged_mla_decode_09_gb300.build import build_library

P = ctypes.c_void_p(256)
BEHIND = (-4, -5, -6)  # workspace too small, no CUDA, another device: the checks of arguments have passed


@pytest.fixture(scope="module")
def lib():
    build_library()
    return mla.load_library()


def prefill(lib, kv_dtype, scale, kv_scale):
    d = mla.MlaPrefillDims(batch=2, num_heads=16, total_q=10, page_size=64, num_pages=16, max_pages_per_req=5,
                           page_table_stride=5, kv_dtype=kv_dtype)
    return lib.mla_prefill(ctypes.byref(d), *[P] * 6, 0, 0, scale, kv_scale, P, P, P, 0, None)


def window(lib, kv_dtype, scale, kv_scale):
    d = mla.MlaDims(batch=2, num_heads=16, q_len=1, page_size=64, num_pages=16, max_pages_per_req=5,
                    page_table_stride=5, kv_dtype=kv_dtype)
    return lib.mla_decode_window(ctypes.byref(d), *[P] * 5, 8, 0, scale, kv_scale, P, P, P, 0, None)


def mass(lib, kv_dtype, scale, kv_scale):
    d = mla.MlaDims(batch=2, num_heads=16, q_len=1, page_size=64, num_pages=16, max_pages_per_req=5,
                    page_table_stride=5, kv_dtype=kv_dtype)
    return lib.mla_attn_mass(ctypes.byref(d), *[P] * 6, 1, scale, kv_scale, P, P, 320, P, 0, None)


@pytest.mark.parametrize("call", [prefill, window, mass])
def test_score_factor(lib, call):
    for scale, kv_scale in ((1e-30, 1e-30), (1e30, 1e30), (3e38, 1.0)):
        assert call(lib, 1, scale, kv_scale) == -1
    assert call(lib, 0, 3e38, 1.0) == -1
    assert call(lib, 1, 1e-20, 1e-20) in BEHIND
    assert call(lib, 1, 0.07, 1e-13) in BEHIND
    assert call(lib, 0, 1e-30, 1e-30) in BEHIND  # a bf16 cache ignores kv_scale
