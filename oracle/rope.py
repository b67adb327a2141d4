"""Rotary positions with the cache write of a step's rows, float64 (test
infrastructure).  The pair (a, b) of a vector's rotated part turns by
position * frequency radians: (a cos - b sin, a sin + b cos), times an
amplitude; pairs are neighbours (interleaved) or half the rotated part apart.
"""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies_ref(rotary_dim, base, factor=1.0, original_len=0, fast=32.0, slow=1.0):
    out = []
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        if factor == 1.0:
            out.append(f)
            continue
        keep = 0.0
        if original_len:
            keep = min(1.0, max(0.0, (original_len * f / (2.0 * math.pi) - slow) / (fast - slow)))
        out.append(keep * f + (1.0 - keep) * f / factor)
    return out


def rope_frequencies_by_index_ref(rotary_dim, base, factor, original_len, fast=32.0, slow=1.0):
    """Between the indices that turn `fast` and `slow` times (rounded outwards),
    the share that is kept falls linearly with the pair's index."""
    def index_of(turns):
        return rotary_dim * math.log(original_len / (2.0 * math.pi * turns)) / (2.0 * math.log(base))

    lo, hi = max(math.floor(index_of(fast)), 0), min(math.ceil(index_of(slow)), rotary_dim - 1)
    out = []
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        keep = min(1.0, max(0.0, (hi - i) / (hi - lo))) if hi > lo else float(i <= lo)
        out.append(f * (keep + (1.0 - keep) / factor))
    return out


def rotate_ref(x, positions, frequencies, interleaved, amplitude=1.0):
    """x float64 [T, ..., n] with its first 2 len(frequencies) values rotated.
    The angle is reduced exactly: its turns are formed as integers over 2^60."""
    y = np.array(x, dtype=np.float64, copy=True)
    r = 2 * len(frequencies)
    for t, p in enumerate(positions):
        for i, f in enumerate(frequencies):
            num, den = (f / (2.0 * math.pi)).as_integer_ratio()
            turn = ((int(p) * num) % den) / den
            c, s = amplitude * math.cos(2.0 * math.pi * turn), amplitude * math.sin(2.0 * math.pi * turn)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, r // 2 + i)
            y[t, ..., a] = x[t, ..., a] * c - x[t, ..., b] * s
            y[t, ..., b] = x[t, ..., a] * s + x[t, ..., b] * c
    return y


def new_slots(page_table, seq_lens, cu_q_lens, page_size=64):
    """(page, row) of every new token, in order."""
    out = []
    for b in range(len(seq_lens)):
        n = int(cu_q_lens[b + 1] - cu_q_lens[b])
        for i in range(n):
            t = int(seq_lens[b]) - n + i
            out.append((int(page_table[b, t // page_size]), t % page_size))
    return out
