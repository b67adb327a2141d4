"""Accumulated attention weight and eviction by it, float64 (test
infrastructure).

Mass: every cached token's sum, over a step's query positions and heads that
see it, of exp(score - lse); a request's q_len queries are its last q_len
tokens, each sees the tokens up to its own position.

Eviction: a request of L tokens keeps k = min(L, budget).  Firm tokens (a
position below num_sinks, or among the num_recent positions that end with the
request's greatest) come first, then the greater weight (a NaN last), then the
lower slot.  A kept token below slot k stays; the free slots below k receive
the tokens kept behind, both in ascending order.
"""
from __future__ import annotations

import math

import numpy as np

from .chunk import cache_rows_at
from .mla_oracle import bf16_bits_to_f64


def attn_mass_ref(q_nope, q_pe, kv_cache, page_table, seq_lens, lse, num_fresh, scale, kv_scale, kv_dtype, mass):
    """Returns float64 mass_out [B, cols]; entries from a request's length on
    are mass's.  q_nope uint16 bits [B, Q, H, 512]; lse [B, Q, H]."""
    B, Q, H, _ = q_nope.shape
    out = np.array(mass, dtype=np.float64)
    for b in range(B):
        L = int(seq_lens[b])
        rows = cache_rows_at(kv_cache, page_table[b], np.arange(L), kv_dtype, kv_scale)
        for t in range(max(0, L - num_fresh), L):
            out[b, t] = 0.0
        for i in range(Q):
            n = L - Q + i + 1
            q = np.concatenate([bf16_bits_to_f64(q_nope[b, i]), bf16_bits_to_f64(q_pe[b, i])], axis=-1)
            for h in range(H):
                if lse[b, i, h] == -np.inf:
                    continue
                out[b, :n] += np.exp(rows[:n] @ q[h] * scale - np.float64(lse[b, i, h]))
    return out


def evict_ref(mass, positions, seq_lens, page_table, kv_cache, budget, num_sinks, num_recent, page_size=64):
    """Returns (new_lens, kept, mass_out, positions_out, cache).  positions may
    be None (a token's slot); outputs start as copies of the inputs."""
    B = len(seq_lens)
    pos_in = np.tile(np.arange(mass.shape[1], dtype=np.int32), (B, 1)) if positions is None else np.asarray(positions)
    new_lens = np.zeros(B, dtype=np.int32)
    kept = np.full((B, budget), -1, dtype=np.int32)
    mass_out, pos_out, cache = np.array(mass), np.array(pos_in), np.array(kv_cache)
    for b in range(B):
        L = int(seq_lens[b])
        k = min(L, budget)
        new_lens[b] = k
        top = max((int(pos_in[b, t]) for t in range(L)), default=0)

        def rank(t):
            p, w = int(pos_in[b, t]), float(mass[b, t])
            if p < num_sinks or p > top - num_recent:
                return (0, 0.0, t)
            return (2, 0.0, t) if math.isnan(w) else (1, -w, t)

        chosen = set(sorted(range(L), key=rank)[:k])
        behind = [t for t in range(k, L) if t in chosen]
        for t in range(k):
            o = t if t in chosen else behind.pop(0)
            kept[b, t], mass_out[b, t], pos_out[b, t] = o, mass[b, o], pos_in[b, o]
            if o != t:
                cache[page_table[b, t // page_size], t % page_size] = \
                    kv_cache[page_table[b, o // page_size], o % page_size]
        assert not behind
    return new_lens, kept, mass_out, pos_out, cache
