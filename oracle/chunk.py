"""Attention of chunks of new tokens over the paged cache, with an optional
sliding window and first tokens that stay visible, float64 (test
infrastructure).

A request's n new tokens are the last n of its L cached ones.  Token i, at
position p = L - n + i, sees the keys t <= p; with a window of w >= 1 tokens
only those with t > p - w, and the first num_sinks tokens.  The attention
over the seen keys is the plain one of mla_oracle.attend.  Only pages that
hold a seen key are looked up.
"""
from __future__ import annotations

import numpy as np

from .mla_oracle import D_LATENT, attend, bf16_bits_to_f64, decode_cache_rows


def seen_keys(pos: int, window: int, num_sinks: int) -> np.ndarray:
    """Positions of the keys that the token at position ``pos`` sees."""
    t = np.arange(pos + 1)
    if window == 0:
        return t
    return t[(t > pos - window) | (t < num_sinks)]


def cache_rows_at(kv_cache, page_table_row, positions, kv_dtype, kv_scale, page_size=64):
    """float64 rows of the given token positions of one request."""
    pages = np.asarray(page_table_row)[positions // page_size]
    if np.any((pages < 0) | (pages >= kv_cache.shape[0])):
        raise IndexError("a page id outside the pool")
    return decode_cache_rows(kv_cache[pages, positions % page_size], kv_dtype, kv_scale)


def mla_prefill_ref(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, window=0, num_sinks=0, scale=1.0,
                    kv_scale=1.0, kv_dtype="bf16"):
    """Returns (out float64 [T, H, 512], lse float64 [T, H]).  q_nope uint16
    bf16 bits [T, H, 512], q_pe [T, H, 64]; rows of tokens that belong to no
    request stay NaN."""
    T, H, _ = q_nope.shape
    out = np.full((T, H, D_LATENT), np.nan)
    lse = np.full((T, H), np.nan)
    for b in range(len(seq_lens)):
        q0, q1 = int(cu_q_lens[b]), int(cu_q_lens[b + 1])
        for i in range(q1 - q0):
            pos = int(seq_lens[b]) - (q1 - q0) + i
            keys = seen_keys(pos, window, num_sinks)
            rows = cache_rows_at(kv_cache, page_table[b], keys, kv_dtype, kv_scale)
            q = np.concatenate([bf16_bits_to_f64(q_nope[q0 + i]), bf16_bits_to_f64(q_pe[q0 + i])], axis=-1)
            out[q0 + i], lse[q0 + i] = attend(q, rows, rows.shape[0], scale)
    return out, lse
