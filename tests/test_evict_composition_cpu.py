"""Why the headers keep windows, attention mass and eviction apart, on the
oracle (no GPU)."""
import os

import numpy as np

import chunk_cases as K
import oracle

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


def _mass(c, lse):
    start = np.zeros((1, 256))
    return oracle.attn_mass_ref(c.q_nope[None], c.q_pe[None], c.kv_cache, c.page_table, c.seq_lens, lse[None], 0,
                                c.scale, 1.0, "bf16", start)[0]


def _attend(c, window, sinks):
    return oracle.mla_prefill_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, window, sinks, c.scale)


def test_weights_add_up_without_a_window_only():
    c = K.make([2], [200], heads=4, seed=1)
    assert np.isclose(_mass(c, _attend(c, 0, 0)[1]).sum(), 8.0, atol=1e-9)
    assert _mass(c, _attend(c, 16, 0)[1]).sum() > 12.0


def test_an_evicted_cache_is_attended_to_without_a_window():
    c = K.make([1], [200], heads=4, seed=2)
    c.kv_cache[c.page_table[0, 3], 8:] = 0
    rng = np.random.default_rng(3)
    mass = rng.random((1, 256)).astype(np.float32)
    n, kept, _, pos, cache = oracle.evict_ref(mass, None, c.seq_lens, c.page_table, c.kv_cache, 100, 0, 30)
    after = K.Chunk(c.q_nope, c.q_pe, cache, c.page_table, n, c.cu, 0, 0, "bf16", 1.0, c.scale)
    rows = oracle.cache_rows_at(c.kv_cache, c.page_table[0], np.sort(kept[0]), "bf16", 1.0)
    q = np.concatenate([oracle.bf16_bits_to_f64(c.q_nope[0]), oracle.bf16_bits_to_f64(c.q_pe[0])], axis=-1)
    want, lse = oracle.attend(q, rows, 100, c.scale)
    out, got = _attend(after, 0, 0)  # the same tokens in another order
    assert np.allclose(out[0], want, atol=1e-12) and np.allclose(got[0], lse, atol=1e-12)
    # the last slots are not the latest positions
    assert set(pos[0, 90:100].tolist()) != set(np.sort(pos[0, :100])[90:].tolist())


def test_the_headers_say_so():
    with open(os.path.join(INCLUDE, "mla_evict.h")) as f:
        text = " ".join(f.read().replace("\n *", " ").split())
    assert "mla_evict and windows. After an eviction a slot is no longer a position" in text
    assert "A windowed or top-k step (mla_decode_window, mla_prefill with a window, mla_decode_sparse) and mla_attn_mass" in text
    with open(os.path.join(INCLUDE, "mla_prefill.h")) as f:
        text = " ".join(f.read().replace("\n *", " ").split())
    assert "slots are no longer positions: call without a window there" in text
