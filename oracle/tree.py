"""Trees of drafted tokens over the paged cache, float64 (test infrastructure).

A request's n nodes are the last n of its L cached tokens, node i in slot
L - n + i; its parent comes before it (-1: none).  A node sees the tokens
before the tree, its ancestors and itself.  The verification walks down from
node 0 and keeps the target's distribution: a child with token x, drawn from
q, is accepted with probability min(1, w[x] / (z q[x])) where w is what earlier
rejections left of the target's row and z its sum; a rejection leaves
max(w - z q, 0).  A fixed proposal counts as drawn from the distribution that
is 1 at x.
"""
from __future__ import annotations

import numpy as np

from .chunk import cache_rows_at
from .mla_oracle import D_LATENT, attend, bf16_bits_to_f64


def ancestors(parents, i: int) -> list:
    """Node i and its ancestors, from the root down."""
    line = []
    while i >= 0:
        line.append(i)
        i = int(parents[i])
    return line[::-1]


def tree_keys(total: int, parents, i: int) -> np.ndarray:
    """Slots that node i of a request of ``total`` tokens sees."""
    base = total - len(parents)
    return np.concatenate([np.arange(base), base + np.asarray(ancestors(parents, i))]).astype(np.int64)


def mla_tree_ref(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, parents, scale=1.0, kv_scale=1.0,
                 kv_dtype="bf16"):
    """Returns (out float64 [T, H, 512], lse float64 [T, H]); arguments as for
    mla_prefill_ref, parents [T].  Rows of no request stay NaN."""
    T, H, _ = q_nope.shape
    out, lse = np.full((T, H, D_LATENT), np.nan), np.full((T, H), np.nan)
    for b in range(len(seq_lens)):
        q0, q1 = int(cu_q_lens[b]), int(cu_q_lens[b + 1])
        for i in range(q1 - q0):
            keys = tree_keys(int(seq_lens[b]), parents[q0:q1], i)
            rows = cache_rows_at(kv_cache, page_table[b], keys, kv_dtype, kv_scale)
            q = np.concatenate([bf16_bits_to_f64(q_nope[q0 + i]), bf16_bits_to_f64(q_pe[q0 + i])], axis=-1)
            out[q0 + i], lse[q0 + i] = attend(q, rows, rows.shape[0], scale)
    return out, lse


def verify_ref(target, draft, tokens, parents, cu_q_lens, accept, sample, cols):
    """Returns (path, tokens_out int32 [B, cols], num_out int32 [B])."""
    B = len(sample)
    path, out = np.full((B, cols), -1, np.int32), np.full((B, cols), -1, np.int32)
    num = np.zeros(B, np.int32)
    for b in range(B):
        q0, n = int(cu_q_lens[b]), int(cu_q_lens[b + 1] - cu_q_lens[b])
        if n == 0:
            continue
        kids = {i: [j for j in range(1, n) if parents[q0 + j] == i and 0 <= tokens[q0 + j] < target.shape[1]]
                for i in range(n)}
        line = [0]
        while True:
            cur = line[-1]
            w, z, went = target[q0 + cur].astype(np.float64), 1.0, False
            for j in kids[cur] if len(line) < cols else []:
                x = int(tokens[q0 + j])
                if draft is None:
                    q = np.zeros_like(w)
                    q[x] = 1.0
                else:
                    q = draft[q0 + cur].astype(np.float64)
                if float(accept[q0 + j]) * z * q[x] < w[x]:
                    out[b, len(line) - 1] = x
                    line.append(j)
                    went = True
                    break
                if draft is None:
                    z = max(z - w[x], 0.0)
                    w[x] = 0.0
                else:
                    w = np.maximum(w - z * q, 0.0)
                    z = w.sum()
            if not went:
                break
        if w.sum() <= 0.0:
            w = target[q0 + line[-1]].astype(np.float64)
        c = np.cumsum(w)
        if c[-1] > 0.0:
            out[b, len(line) - 1] = int(np.argmax(c > float(sample[b]) * c[-1]))
        path[b, :len(line)] = line
        num[b] = len(line)
    return path, out, num


def tree_commit_ref(kv_cache, page_table, seq_lens, cu_q_lens, path, num_path, page_size=64):
    """Returns (new cache, new_lens); kv_cache [layers, P, 64, 576]."""
    cache, new_lens = np.array(kv_cache, copy=True), np.array(seq_lens, copy=True)
    for b in range(len(seq_lens)):
        base = int(seq_lens[b]) - int(cu_q_lens[b + 1] - cu_q_lens[b])
        for k in range(int(num_path[b])):
            f, t = base + int(path[b, k]), base + k
            cache[:, page_table[b, t // page_size], t % page_size] = kv_cache[:, page_table[b, f // page_size],
                                                                              f % page_size]
        new_lens[b] = base + int(num_path[b])
    return cache, new_lens
