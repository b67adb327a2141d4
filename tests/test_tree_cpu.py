"""mla_decode_tree, mla_tree_commit and mla_verify without a GPU: refusals of
the C entry points and the binding, and the pins of the oracle that the GPU
tests use."""
import ctypes

import numpy as np
import pytest

import chunk_cases as K
import oracle
import paged_mla_decode_09_gb300 as mla
import tree_cases as TC
from paged_mla_decode_09_gb300.build import build_library


@pytest.fixture(scope="module")
def lib():
    build_library()
    return mla.load_library()


P = ctypes.c_void_p(1 << 20)


def _dims(**kw):
    d = dict(batch=2, num_heads=16, total_q=10, page_size=64, num_pages=16, max_pages_per_req=5, page_table_stride=5,
             kv_dtype=0)
    d.update(kw)
    return mla.MlaPrefillDims(**d)


def _tree(lib, d, ptrs=None, scale=1.0, kv_scale=1.0):
    a = [P] * 10 if ptrs is None else ptrs
    return lib.mla_decode_tree(ctypes.byref(d), *a[:7], scale, kv_scale, *a[7:], 1 << 40, None)


@pytest.mark.parametrize("bad", [dict(batch=0), dict(num_heads=0), dict(total_q=0), dict(num_pages=0),
                                 dict(max_pages_per_req=0), dict(page_table_stride=4)])
def test_tree_refuses_bad_dims(lib, bad):
    assert _tree(lib, _dims(**bad)) == -1
    assert lib.mla_decode_tree_workspace_size(ctypes.byref(_dims(**bad)), 0) == 0


@pytest.mark.parametrize("bad", [dict(page_size=32), dict(kv_dtype=2), dict(total_q=1 << 28), dict(num_pages=1 << 26),
                                 dict(max_pages_per_req=1 << 26, page_table_stride=1 << 26)])
def test_tree_refuses_what_it_does_not_support(lib, bad):
    assert _tree(lib, _dims(**bad)) == -2
    assert lib.mla_decode_tree_workspace_size(ctypes.byref(_dims(**bad)), 0) == 0


def test_tree_refuses_bad_arguments(lib):
    d = _dims()
    for k in range(10):
        ptrs = [P] * 10
        ptrs[k] = None
        assert _tree(lib, d, ptrs) == -1, k
    for k, off in ((0, 16), (1, 16), (2, 8), (3, 2), (4, 2), (5, 2), (6, 2), (7, 16), (8, 2), (9, 128)):
        ptrs = [P] * 10
        ptrs[k] = ctypes.c_void_p((1 << 20) + off)
        assert _tree(lib, d, ptrs) == -3, k
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _tree(lib, d, scale=s) == -1
        assert _tree(lib, _dims(kv_dtype=1), kv_scale=s) == -1


def _commit(lib, ptrs=None, **kw):
    d = dict(batch=2, num_layers=1, path_cols=4, num_pages=16, max_pages_per_req=5, page_table_stride=5, kv_dtype=0,
             reserved=0, layer_stride=0)
    d.update(kw)
    a = [ctypes.c_void_p((k + 1) << 20) for k in range(8)] if ptrs is None else ptrs
    return lib.mla_tree_commit(ctypes.byref(mla.MlaTreeCommitDims(**d)), *a, None)


def test_commit_refusals(lib):
    for bad in (dict(batch=0), dict(num_layers=0), dict(path_cols=0), dict(num_pages=0), dict(max_pages_per_req=0),
                dict(page_table_stride=4), dict(num_layers=2, layer_stride=16 * 64 * 1152 - 16)):
        assert _commit(lib, **bad) == -1, bad
    for bad in (dict(kv_dtype=3), dict(batch=65536), dict(num_layers=65536, layer_stride=1 << 40),
                dict(num_pages=1 << 25), dict(max_pages_per_req=1 << 25, page_table_stride=1 << 25)):
        assert _commit(lib, **bad) == -2, bad
    assert _commit(lib, num_layers=2, layer_stride=16 * 64 * 1152 + 8) == -3
    good = [ctypes.c_void_p((k + 1) << 20) for k in range(8)]
    for k in range(8):
        assert _commit(lib, good[:k] + [None] + good[k + 1:]) == -1, k
        off = ctypes.c_void_p(((k + 1) << 20) + (8 if k == 0 else 2))
        assert _commit(lib, good[:k] + [off] + good[k + 1:]) == -3, k
    # new lengths over what every block reads
    for k in (2, 3, 5):
        assert _commit(lib, good[:6] + [good[k]] + good[7:]) == -1
    assert _commit(lib, good[:6] + [ctypes.c_void_p(good[2].value + 4)] + good[7:]) == -1
    assert lib.mla_tree_commit(None, *good, None) == -1


def test_commit_refuses_outputs_over_inputs(lib):
    """New lengths and the status word over each buffer that every block reads,
    from its first and over its last element; 2 requests, 4 path columns, 5 pages."""
    # (the cache is off its alignment, which is looked at next: no call gets further)
    good = [ctypes.c_void_p((1 << 20) + 8)] + [ctypes.c_void_p((k + 1) << 20) for k in range(1, 8)]
    assert _commit(lib, good) == -3
    words = {1: 2 * 5, 2: 2, 3: 3, 4: 2 * 4, 5: 2, 6: 2, 7: 1}
    for out in (6, 7):
        for other in words:
            if other != out:
                for at in (0, words[other] - 1):
                    a = list(good)
                    a[out] = ctypes.c_void_p(a[other].value + 4 * at)
                    assert _commit(lib, a) == -1, (out, other, at)
                a[out] = ctypes.c_void_p(a[other].value + 4 * words[other])  # right behind it
                assert _commit(lib, a) == -3, (out, other)
    # rows of 5 entries, 9 apart: in the gap, at its end, one further, behind the last row
    for at, rc in ((4, -1), (5, -3), (7, -3), (8, -1), (9, -1), (14, -3)):
        a = list(good)
        a[6] = ctypes.c_void_p(a[1].value + 4 * at)
        assert _commit(lib, a, page_table_stride=9) == rc, at


V = [ctypes.c_void_p((k + 1) << 20) for k in range(11)]


def _verify(lib, ptrs=None, **kw):
    d = dict(batch=2, total_q=6, vocab=100, path_cols=4, target_stride=100, draft_stride=100)
    d.update(kw)
    a = V if ptrs is None else ptrs
    return lib.mla_verify(ctypes.byref(mla.MlaVerifyDims(**d)), *a, None)


def test_verify_refusals(lib):
    for bad in (dict(batch=0), dict(total_q=0), dict(vocab=0), dict(path_cols=0), dict(target_stride=99),
                dict(draft_stride=99)):
        assert _verify(lib, **bad) == -1, bad
    for bad in (dict(vocab=(1 << 20) + 1, target_stride=1 << 21, draft_stride=1 << 21), dict(batch=(1 << 27) + 1),
                dict(target_stride=1 << 41)):
        assert _verify(lib, **bad) == -2, bad
    def but(k, p):
        return V[:k] + [p] + V[k + 1:]

    for k in range(11):
        if k != 1:  # no draft: fixed proposals
            assert _verify(lib, but(k, None)) == -1, k
        assert _verify(lib, but(k, ctypes.c_void_p(V[k].value + 2))) == -3, k
    # without a draft its stride is not looked at: what is refused is the next thing
    assert _verify(lib, [V[0], None, ctypes.c_void_p(V[2].value + 2)] + V[3:], draft_stride=0) == -3
    assert lib.mla_verify(None, *V, None) == -1
    # outputs over inputs or one another
    for out in range(7, 11):
        for other in [2, 3, 4, 5, 6] + [k for k in range(7, 11) if k != out]:
            assert _verify(lib, but(out, V[other])) == -1, (out, other)


def test_verify_refuses_outputs_over_probabilities(lib):
    """6 rows of 100 entries, 104 apart.  (tokens is off its alignment, which is
    looked at next: no call gets further.)"""
    good = V[:2] + [ctypes.c_void_p(V[2].value + 2)] + V[3:]
    wide = dict(target_stride=104, draft_stride=104)
    assert _verify(lib, good, **wide) == -3
    for out, n in ((7, 8), (8, 8), (9, 2), (10, 1)):
        for rows in (0, 1):
            for at, rc in ((0, -1), (100 - n, -1), (99, -1), (5 * 104 + 99, -1), (5 * 104 + 100, -3),
                           (100, -3 if n <= 4 else -1), (104 - n, -3 if n <= 4 else -1), (105 - n, -1)):
                a = list(good)
                a[out] = ctypes.c_void_p(a[rows].value + 4 * at)
                assert _verify(lib, a, **wide) == rc, (out, rows, at)
    a = list(good)  # no draft: its place is free
    a[1], a[7] = None, V[1]
    assert _verify(lib, a, **wide) == -3


def test_binding_refuses_what_the_library_cannot_see(lib):
    torch = pytest.importorskip("torch")
    z = torch.zeros
    cache, table, lens = z(4, 64, 576, dtype=torch.bfloat16), z(2, 2, dtype=torch.int32), z(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors
        mla.mla_tree_commit(cache, table, lens, z(3, dtype=torch.int32), z(2, 4, dtype=torch.int32), lens, lens, lens)
    with pytest.raises(ValueError):
        mla.mla_verify(z(6, 10), None, z(6), z(6), z(3), z(6), z(2), z(2, 4), z(2, 4), z(2), z(1))
    with pytest.raises(ValueError):
        mla.mla_decode_tree(*[z(2, 3, 4)] * 7, 1.0, 1.0, z(2), z(2), z(2))
    # layouts (looked at on any device)
    assert mla._layers_of(cache) == (1, 4, 0)
    many = z(3, 4, 64, 576, dtype=torch.uint8)
    assert mla._layers_of(many) == (3, 4, 4 * 64 * 576)
    assert mla._layers_of(z(3, 8, 64, 576, dtype=torch.uint8)[:, :4]) == (3, 4, 8 * 64 * 576)
    for bad in (cache.float(), cache[:, :32], cache[..., :512], many[:, ::2], many.transpose(0, 1), cache[0]):
        with pytest.raises(ValueError):
            mla._check_layers(bad)
    with pytest.raises(ValueError):
        mla._check_probs("target", z(6, 10).double(), 6, 10)
    with pytest.raises(ValueError):
        mla._check_probs("target", z(10, 6).t(), 6, 10)
    with pytest.raises(ValueError):
        mla._check_probs("target", z(1, 10).expand(6, 10), 6, 10)
    mla._check_probs("target", z(6, 12)[:, :10], 6, 10)


# ---- the oracle ----

def test_tree_keys_by_hand():
    parents = [-1, 0, 0, 1, -1, 3]
    assert oracle.tree_keys(8, parents, 0).tolist() == [0, 1, 2]
    assert oracle.tree_keys(8, parents, 2).tolist() == [0, 1, 2, 4]
    assert oracle.tree_keys(8, parents, 5).tolist() == [0, 1, 2, 3, 5, 7]
    assert oracle.tree_keys(6, parents, 4).tolist() == [4]


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_oracle_chain_is_the_prompt_chunk(kv_dtype):
    c, parents = TC.make([3, 0, 5], [70, 3, 130], heads=3, kind="chain", kv_dtype=kv_dtype, seed=2)
    a = oracle.mla_tree_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, parents, c.scale, c.kv_scale,
                            kv_dtype)
    b = oracle.mla_prefill_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, 0, 0, c.scale, c.kv_scale,
                               kv_dtype)
    assert np.allclose(a[0], b[0], rtol=0, atol=1e-12) and np.allclose(a[1], b[1], rtol=0, atol=1e-12)


def test_oracle_node_is_its_own_branch_alone():
    """A node's output is that of a request whose last tokens are its branch."""
    c, parents = TC.make([9], [100], heads=2, seed=5)
    out, lse = oracle.mla_tree_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, parents, c.scale)
    rows = oracle.bf16_bits_to_f64(c.kv_cache[c.page_table[0]].reshape(-1, 576))
    for i in range(9):
        line, at = [], i
        while at >= 0:
            line, at = [91 + at] + line, parents[at]
        k = np.concatenate([rows[:91], rows[line]])
        q = np.concatenate([oracle.bf16_bits_to_f64(c.q_nope[i]), oracle.bf16_bits_to_f64(c.q_pe[i])], axis=1)
        w = np.exp(q @ k.T * c.scale)
        assert np.allclose(lse[i], np.log(w.sum(axis=1)), atol=1e-12)
        assert np.allclose(out[i], (w / w.sum(axis=1, keepdims=True)) @ k[:, :512], atol=1e-12)


def test_verify_by_hand():
    """Numbers with few bits: every comparison is exact."""
    p = np.array([[0.5, 0.25, 0.25, 0.0], [0.25, 0.25, 0.0, 0.5], [1.0, 0.0, 0.0, 0.0]], np.float32)
    q = np.array([[0.25, 0.25, 0.5, 0.0], [0.0, 0.5, 0.0, 0.5], [0.25] * 4], np.float32)
    cu, chain = [0, 3], [-1, 0, 1]

    def one(draft, tokens, parents, accept, sample, cols=3):
        path, out, num = oracle.verify_ref(p, draft, tokens, parents, cu, accept, [sample], cols)
        return path[0, :num[0]].tolist(), out[0, :num[0]].tolist()

    # node 1 (token 2, p 0.25, q 0.5): accepted below 0.5; node 2 (token 3, p = q): always
    assert one(q, [0, 2, 3], chain, [0, 0.4375, 0.9375], 0.0) == ([0, 1, 2], [2, 3, 0])
    # rejected at 0.5 itself: what is left of p - q is 0.25 at token 0
    assert one(q, [0, 2, 3], chain, [0, 0.5, 0.0], 0.9375) == ([0], [0])
    # two children of node 0: the second after max(p - q, 0) = [0.25, 0, 0, 0]
    assert one(q, [0, 2, 0], [-1, 0, 0], [0, 0.75, 0.5], 0.0) == ([0, 2], [0, 0])
    # (z = 0.25, q = 0.25 at token 0: accepted at any number below 4, so always)
    # fixed proposals: 1 (0.25), then 0 (0.5 of the 0.75 left), then the rest
    assert one(None, [0, 1, 0], [-1, 0, 0], [0, 0.125, 0.0], 0.5) == ([0, 1], [1, 3])
    assert one(None, [0, 1, 0], [-1, 0, 0], [0, 0.25, 0.625], 0.5) == ([0, 2], [0, 0])
    assert one(None, [0, 1, 0], [-1, 0, 0], [0, 0.25, 0.75], 0.5) == ([0], [2])
    # the same token twice: nothing is left for the second
    assert one(None, [0, 1, 1], [-1, 0, 0], [0, 0.25, 0.0], 0.0) == ([0], [0])
    # a full row ends the walk
    assert one(q, [0, 2, 3], chain, [0, 0.0, 0.0], 0.0, cols=1) == ([0], [0])
    # the borders of the last token: sums 0.5, 0.75, 1
    assert [one(None, [0, 0, 0], [-1, -1, -1], [0, 0, 0], s)[1][0] for s in (0.0, 0.4375, 0.5, 0.6875, 0.75, 0.9375)] \
        == [0, 0, 1, 1, 2, 2]


@pytest.mark.parametrize("drafted", [True, False])
def test_verified_tokens_are_distributed_as_the_target(drafted):
    """First tokens of many requests against the target's row: counts within
    five standard deviations (sqrt(n p (1 - p)) of a binomial)."""
    rng = np.random.default_rng(3)
    n, v = 20000, 5
    p = rng.dirichlet(np.ones(v)).astype(np.float32)
    q = rng.dirichlet(np.ones(v)).astype(np.float32)
    nodes = 4
    parents = [-1, 0, 0, 0] * n
    tokens = np.zeros(n * nodes, np.int64)
    for b in range(n):
        tokens[b * nodes + 1:b * nodes + 4] = (rng.choice(v, 3, p=q / q.astype(np.float64).sum()) if drafted
                                               else [3, 0, 4])
    rows = np.broadcast_to(p, (n * nodes, v))
    draft = np.broadcast_to(q, (n * nodes, v)) if drafted else None
    _, out, _ = oracle.verify_ref(rows, draft, tokens, parents, np.arange(n + 1) * nodes, rng.random(n * nodes),
                                  rng.random(n), 2)
    counts = np.bincount(out[:, 0], minlength=v)
    pp = p.astype(np.float64) / p.sum(dtype=np.float64)
    assert np.all(np.abs(counts - n * pp) <= 5 * np.sqrt(n * pp * (1 - pp)))


def test_commit_ref_by_hand():
    cache = np.arange(2 * 3 * 64, dtype=np.uint16).reshape(2, 3, 64, 1).repeat(576, axis=3)
    table = np.array([[2, 0]], np.int32)
    new, lens = oracle.tree_commit_ref(cache, table, [66], [0, 5], np.array([[0, 2, 4, -1]]), [3])
    assert lens.tolist() == [64]
    assert new[0, 2, 61, 0] == cache[0, 2, 61, 0]
    assert new[0, 2, 62, 0] == cache[0, 2, 63, 0] and new[1, 2, 63, 0] == cache[1, 0, 1, 0]
    assert np.array_equal(new[:, 0], cache[:, 0]) and np.array_equal(new[:, 1], cache[:, 1])
