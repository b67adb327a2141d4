"""mla_attn_mass and mla_evict without a GPU: refusals of the C entry points
and the binding, and pins of the oracle that the GPU tests use."""
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
    d = dict(batch=2, num_heads=16, q_len=1, page_size=64, num_pages=16, max_pages_per_req=5, page_table_stride=5,
             kv_dtype=0)
    d.update(kw)
    return mla.MlaDims(**d)


def _edims(**kw):
    d = dict(batch=2, mass_cols=320, num_pages=16, max_pages_per_req=5, page_table_stride=5, kv_dtype=0, budget=64,
             num_sinks=4, num_recent=8)
    d.update(kw)
    return mla.MlaEvictDims(**d)


def _mass(lib, d, ptrs=None, fresh=1, scale=1.0, kv_scale=1.0, cols=320, ws=256):
    a = [P] * 9 if ptrs is None else ptrs  # q_nope q_pe cache table lens lse mass mass_out workspace
    return lib.mla_attn_mass(ctypes.byref(d), *a[:6], fresh, scale, kv_scale, a[6], a[7], cols, a[8], ws, None)


def _evict(lib, d, ptrs=None, ws=1 << 40):
    a = [P] * 10 if ptrs is None else ptrs  # mass pos lens table cache new_lens kept mass_out pos_out workspace
    return lib.mla_evict(ctypes.byref(d), *a, ws, None)


@pytest.mark.parametrize("bad,rc", [
    (dict(batch=0), -1), (dict(num_heads=0), -1), (dict(q_len=0), -1), (dict(num_pages=0), -1),
    (dict(max_pages_per_req=0), -1), (dict(page_table_stride=4), -1), (dict(page_size=32), -2), (dict(kv_dtype=9), -2),
    (dict(num_pages=1 << 26), -2), (dict(batch=1 << 14, max_pages_per_req=1 << 12, page_table_stride=1 << 12), -2),
    (dict(batch=1, max_pages_per_req=(1 << 24) + 1, page_table_stride=1 << 25), -2),
    (dict(batch=1 << 20, q_len=1 << 11), -2), (dict(batch=1 << 12, q_len=1 << 10, num_heads=1 << 10), -2)])
def test_mass_refuses_dims(lib, bad, rc):
    assert _mass(lib, _dims(**bad)) == rc
    assert lib.mla_attn_mass_workspace_size(ctypes.byref(_dims(**bad)), 0) == 0


def test_mass_refuses_arguments(lib):
    d = _dims()
    assert lib.mla_attn_mass_workspace_size(ctypes.byref(d), 0) == 256
    for k in (0, 1, 2, 3, 4, 5, 7, 8):
        ptrs = [P] * 9
        ptrs[k] = None
        assert _mass(lib, d, ptrs) == -1, k
    for k, off in ((0, 16), (1, 16), (2, 8), (3, 2), (4, 2), (5, 2), (6, 2), (7, 2), (8, 128)):
        ptrs = [P] * 9
        ptrs[k] = ctypes.c_void_p(256 + off)
        assert _mass(lib, d, ptrs) == -3, k
    assert _mass(lib, d, fresh=-1) == -1
    assert _mass(lib, d, cols=0) == -1
    assert _mass(lib, d, ws=255) == -4
    for s in (0.0, -2.0, float("nan"), float("inf")):
        assert _mass(lib, d, scale=s) == -1
        assert _mass(lib, _dims(kv_dtype=1), kv_scale=s) == -1


@pytest.mark.parametrize("bad,rc", [
    (dict(batch=0), -1), (dict(mass_cols=0), -1), (dict(num_pages=0), -1), (dict(max_pages_per_req=0), -1),
    (dict(page_table_stride=4), -1), (dict(budget=0), -1), (dict(num_sinks=-1), -1), (dict(num_recent=-1), -1),
    (dict(num_sinks=60, num_recent=5), -1), (dict(num_sinks=2**31 - 1, num_recent=2**31 - 1), -1),
    (dict(kv_dtype=3), -2), (dict(num_pages=1 << 26), -2), (dict(batch=65536), -2),
    (dict(mass_cols=(1 << 30) + 1), -2), (dict(budget=(1 << 30) + 1), -2),
    (dict(max_pages_per_req=1 << 26, page_table_stride=1 << 26), -2)])
def test_evict_refuses_dims(lib, bad, rc):
    assert _evict(lib, _edims(**bad)) == rc


def test_evict_refuses_arguments(lib):
    d = _edims()
    for k in (0, 2, 3, 4, 5, 6, 7, 8, 9):
        ptrs = [P] * 10
        ptrs[k] = None
        assert _evict(lib, d, ptrs) == -1, k  # positions_out (8) is needed with positions
    for k, off in ((0, 2), (1, 2), (2, 2), (3, 2), (4, 8), (5, 2), (6, 2), (7, 2), (8, 2), (9, 128)):
        ptrs = [P] * 10
        ptrs[k] = ctypes.c_void_p(256 + off)
        assert _evict(lib, d, ptrs) == -3, k
    assert lib.mla_evict_workspace_size(0, 5) == 0 and lib.mla_evict_workspace_size(5, 0) == 0
    n = lib.mla_evict_workspace_size(2, 64)
    assert n >= 2 * 64 * 8
    assert _evict(lib, d, ws=n - 1) == -4


def test_binding_layout_checks():
    torch = pytest.importorskip("torch")
    c = K.make([2, 2], [70, 100], heads=4, seed=1)
    bf = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16)  # noqa: E731
    m = dict(q_nope=bf(c.q_nope).view(2, 2, 4, 512), q_pe=bf(c.q_pe).view(2, 2, 4, 64), kv_cache=bf(c.kv_cache),
             page_table=torch.from_numpy(c.page_table), seq_lens=torch.from_numpy(c.seq_lens),
             lse=torch.zeros(2, 2, 4), mass=torch.zeros(2, 128), mass_out=torch.zeros(2, 128),
             workspace=torch.zeros(256, dtype=torch.uint8))
    mla._check_mass_tensors(**m)
    mla._check_mass_tensors(**{**m, "mass": None})
    for name, x in (("lse", torch.zeros(2, 2, 4).double()), ("mass", torch.zeros(2, 64)), ("mass", torch.zeros(2, 256)[:, ::2]),
                    ("mass_out", torch.zeros(256)), ("q_nope", m["q_nope"][0]), ("seq_lens", m["seq_lens"].long()),
                    ("mass_out", torch.zeros(3, 128))):
        with pytest.raises((ValueError, TypeError)):
            mla._check_mass_tensors(**{**m, name: x})
    i32 = dict(dtype=torch.int32)
    e = dict(mass=m["mass"], positions=torch.zeros(2, 128, **i32), seq_lens=m["seq_lens"], page_table=m["page_table"],
             kv_cache=m["kv_cache"], budget=64, new_lens=torch.zeros(2, **i32), kept=torch.zeros(2, 64, **i32),
             mass_out=m["mass_out"], positions_out=torch.zeros(2, 128, **i32), workspace=m["workspace"])
    mla._check_evict_tensors(**e)
    mla._check_evict_tensors(**{**e, "positions": None, "positions_out": None})
    for name, x in (("positions", torch.zeros(2, 128)), ("positions_out", None), ("kept", torch.zeros(2, 63, **i32)),
                    ("new_lens", torch.zeros(2)), ("mass", torch.zeros(128)), ("mass_out", torch.zeros(2, 64)),
                    ("kv_cache", m["kv_cache"][:, :32].contiguous()), ("page_table", m["page_table"][:1])):
        with pytest.raises((ValueError, TypeError)):
            mla._check_evict_tensors(**{**e, name: x})
    with pytest.raises(ValueError):
        mla.mla_evict(e["mass"], None, e["seq_lens"], e["page_table"], e["kv_cache"], 64, 0, 0, e["new_lens"],
                      e["kept"], e["mass_out"], None, e["workspace"])  # CPU tensors


# ---- the oracle ----

def test_evict_oracle_by_hand():
    mass = np.array([[1, 9, 2, 8, 3, 7, 4, 6, 0, 0]], dtype=np.float32)
    table = np.array([[0]], dtype=np.int32)
    cache = np.arange(64, dtype=np.uint8)[None, :, None].repeat(576, axis=2)
    n, kept, mo, po, out = oracle.evict_ref(mass, None, np.array([8]), table, cache, 5, 0, 0)
    # weights 9 8 7 6 4 stay: slots 1 3 5 7 6; slots 0 2 4 are free and get 5 6 7
    assert n.tolist() == [5] and kept[0].tolist() == [5, 1, 6, 3, 7]
    assert mo[0, :5].tolist() == [7, 9, 4, 8, 6] and po[0, :5].tolist() == [5, 1, 6, 3, 7]
    assert out[0, :8, 0].tolist() == [5, 1, 6, 3, 7, 5, 6, 7]
    # the first token and the two latest positions are firm
    n, kept, *_ = oracle.evict_ref(mass, None, np.array([8]), table, cache, 4, 1, 2)
    assert kept[0].tolist() == [0, 1, 6, 7]
    pos = np.array([[0, 50, 51, 9, 8, 7, 6, 5, 99, 99]], dtype=np.int32)  # slots 1 and 2 are the latest
    n, kept, *_ = oracle.evict_ref(mass, pos, np.array([8]), table, cache, 4, 0, 2)
    assert kept[0].tolist() == [5, 1, 2, 3]
    # nothing to do within the budget
    n, kept, *_ = oracle.evict_ref(mass, None, np.array([3]), table, cache, 5, 0, 0)
    assert n.tolist() == [3] and kept[0].tolist() == [0, 1, 2, -1, -1]


def test_evict_oracle_keeps_the_best_set():
    rng = np.random.default_rng(0)
    mass = rng.random((1, 192)).astype(np.float32)
    table = np.array([[2, 0, 1]], dtype=np.int32)
    cache = rng.integers(0, 255, size=(3, 64, 576)).astype(np.uint8)
    n, kept, mo, _, out = oracle.evict_ref(mass, None, np.array([150]), table, cache, 70, 0, 0)
    assert set(kept[0].tolist()) == set(np.argsort(-mass[0, :150])[:70].tolist())
    for t in range(70):
        o = kept[0, t]
        assert np.array_equal(out[table[0, t // 64], t % 64], cache[table[0, o // 64], o % 64])


def test_mass_oracle_adds_to_one_per_row():
    c = K.make([2], [130], heads=3, seed=3)
    _, lse = oracle.mla_prefill_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, 0, 0, c.scale)
    q, p = c.q_nope.reshape(1, 2, 3, 512), c.q_pe.reshape(1, 2, 3, 64)
    start = np.full((1, 192), 5.0)
    out = oracle.attn_mass_ref(q, p, c.kv_cache, c.page_table, c.seq_lens, lse.reshape(1, 2, 3), 2, c.scale, 1.0, "bf16",
                               start)
    assert np.isclose(out[0, :130].sum(), 128 * 5.0 + 6.0, atol=1e-9)
    assert np.all(out[0, 130:] == 5.0) and out[0, 128] < 5.0 and out[0, 129] < 5.0
    # one query row: its softmax
    one = oracle.attn_mass_ref(q[:, 1:, :1], p[:, 1:, :1], c.kv_cache, c.page_table, c.seq_lens,
                               lse.reshape(1, 2, 3)[:, 1:, :1], 130, c.scale, 1.0, "bf16", start)
    k = oracle.cache_rows_at(c.kv_cache, c.page_table[0], np.arange(130), "bf16", 1.0)
    s = k @ np.concatenate([oracle.bf16_bits_to_f64(q[0, 1, 0]), oracle.bf16_bits_to_f64(p[0, 1, 0])]) * c.scale
    w = np.exp(s - s.max())
    assert np.allclose(one[0, :130], w / w.sum(), atol=1e-12)
