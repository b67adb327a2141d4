"""CPU float64 oracle for paged MLA decode.

TEST INFRASTRUCTURE ONLY. Nothing on the product path may import this
package: only ``tests/``, ``__graft_entry__.smoke()`` and the CPU-baseline /
reference legs of ``bench.py`` use it. It shares no code with the CUDA
library (no kernels, headers, tables or helpers).

Parity status: every public function is pinned by ``tests/test_oracle_pins.py``
against an independent check (non-absorbed attention, closed forms, the
split/merge identity, brute force, and torch's own float8 decoder).
"""
from .chunk import cache_rows_at, mla_prefill_ref, seen_keys
from .e4m3 import e4m3_decode_table, e4m3_encode, e4m3_to_f64
from .evict import attn_mass_ref, evict_ref
from .kv_pack import kv_pack_ref
from .pages import page_fork_ref, page_resize_ref
from .rope import new_slots, rope_frequencies_by_index_ref, rope_frequencies_ref, rotate_ref
from .sparse import mla_decode_sparse_ref
from .tree import ancestors, mla_tree_ref, tree_commit_ref, tree_keys, verify_ref
from .mla_oracle import (
    attend,
    bf16_bits_to_f64,
    decode_cache_rows,
    gather_rows,
    lse_merge,
    mla_decode_ref,
    mla_decode_ref_pieces,
    visible_keys,
)

__all__ = [
    "ancestors",
    "attend",
    "attn_mass_ref",
    "cache_rows_at",
    "e4m3_decode_table",
    "e4m3_encode",
    "e4m3_to_f64",
    "bf16_bits_to_f64",
    "evict_ref",
    "decode_cache_rows",
    "gather_rows",
    "kv_pack_ref",
    "lse_merge",
    "mla_decode_ref",
    "mla_decode_ref_pieces",
    "mla_decode_sparse_ref",
    "mla_prefill_ref",
    "mla_tree_ref",
    "new_slots",
    "page_fork_ref",
    "page_resize_ref",
    "rope_frequencies_by_index_ref",
    "rope_frequencies_ref",
    "rotate_ref",
    "seen_keys",
    "tree_commit_ref",
    "tree_keys",
    "verify_ref",
    "visible_keys",
]
