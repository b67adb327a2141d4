"""Seeded trees of drafted tokens for the tests, and error bounds for nodes."""
import numpy as np

import chunk_cases as K
import oracle


def random_tree(rng, n, near=6, forest=False):
    """Parents of n nodes: mostly one of the few before; a forest has several
    nodes without one."""
    p = [-1]
    for i in range(1, n):
        p.append(-1 if forest and rng.random() < 0.2 else int(rng.integers(max(0, i - near), i)))
    return p[:n]


def make(new, total, heads, kind="tree", seed=0, **kw):
    """A chunk_cases batch and the parents of its nodes, int32 [T] (entries
    behind the last request are garbage)."""
    c = K.make(new, total, heads, seed=seed, **kw)
    rng = np.random.default_rng(seed + 1000)
    parents = []
    for n in new:
        if kind == "chain":
            parents += [i - 1 for i in range(n)]
        elif kind == "star":
            parents += [-1] + [0] * (n - 1) if n else []
        elif kind == "none":
            parents += [-1] * n
        else:
            parents += random_tree(rng, n, forest=kind == "forest") if n else []
    parents += [12345] * (c.q_nope.shape[0] - len(parents))
    return c, np.asarray(parents, dtype=np.int32)


def error_bounds(c, b, i, keys):
    """chunk_cases.error_bounds (the roundings are counted there) for a node
    that sees the given slots."""
    rows = oracle.cache_rows_at(c.kv_cache, c.page_table[b], keys, c.kv_dtype, c.kv_scale)
    t = int(c.cu[b]) + i
    q = np.concatenate([oracle.bf16_bits_to_f64(c.q_nope[t]), oracle.bf16_bits_to_f64(c.q_pe[t])], axis=-1)
    s = (q @ rows.T) * c.scale
    top = s.max(axis=1, keepdims=True)
    w = np.exp(s - top)
    z = w.sum(axis=1, keepdims=True)
    w /= z
    d = 584 * 2.0**-23 * (np.abs(q) @ np.abs(rows).T).max(axis=1) * c.scale
    if c.kv_dtype != "bf16":
        d = d + 2.0**-17 * np.abs(q).max(axis=1) * np.abs(rows).sum(axis=1).max() * c.scale
    acc = (len(keys) / 16 + 64) * 2.0**-23
    ref, mean_abs = w @ rows[:, :512], w @ np.abs(rows[:, :512])
    lse = top[:, 0] + np.log(z[:, 0])
    out_tol = 2.0**-8 * np.abs(ref) + (2.0**-8 + acc + 2 * d)[:, None] * mean_abs + 1e-30
    return ref, lse, out_tol, d + acc + 8 * 2.0**-23 * (np.abs(lse) + 1)
