"""Pages handed out, shared and freed by reference counts (test
infrastructure): plain loops over table rows.  A page with count 0 is free;
free pages go out lowest id first, to the missing entries row by row.
"""
from __future__ import annotations

import numpy as np

NO_PAGES = 512


def _hand_out(table, refs, missing):
    free = [i for i in range(len(refs)) if refs[i] == 0]
    status = NO_PAGES if len(missing) > len(free) else 0
    for (b, c), page in zip(missing, free):
        table[b, c] = page
        refs[page] = 1
    return status


def page_resize_ref(new_lens, page_table, page_refs, page_size=64):
    """Returns (page_table, page_refs, status)."""
    table, refs = np.array(page_table, copy=True), np.array(page_refs, copy=True)
    missing = []
    for b, n in enumerate(new_lens):
        need = -(-int(n) // page_size)
        for c in range(table.shape[1]):
            if c < need:
                if table[b, c] < 0:
                    table[b, c] = -1
                    missing.append((b, c))
            else:
                if table[b, c] >= 0:
                    refs[table[b, c]] -= 1
                table[b, c] = -1
    return table, refs, _hand_out(table, refs, missing)


def page_fork_ref(src, seq_lens, page_table, page_refs, kv_cache, page_size=64):
    """Returns (page_table_out, page_refs, cache, status); kv_cache [layers, P, 64, 576]."""
    refs, cache = np.array(page_refs, copy=True), np.array(kv_cache, copy=True)
    out = np.full((len(src), page_table.shape[1]), -1, np.int32)
    missing = []
    for c, s in enumerate(src):
        if s < 0:
            continue
        full, tail = divmod(int(seq_lens[s]), page_size)
        out[c, :full] = page_table[s, :full]
        for page in page_table[s, :full]:
            refs[page] += 1
        if tail:
            missing.append((c, full))
    status = _hand_out(out, refs, missing)
    for c, full in missing:
        if out[c, full] >= 0:
            s = src[c]
            tail = int(seq_lens[s]) % page_size
            cache[:, out[c, full], :tail] = kv_cache[:, page_table[s, full], :tail]
    return out, refs, cache, status
