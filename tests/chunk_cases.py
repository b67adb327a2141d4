"""Seeded batches for the prompt-chunk, window and attention-mass tests:
ragged lengths, a page table whose unneeded entries are -1, NaN in every slot
that no query may see because it lies behind its sequence."""
from dataclasses import dataclass

import numpy as np

from paged_mla_decode_09_gb300 import workloads as W

SCALE = W.SCALE_192


@dataclass
class Chunk:
    q_nope: np.ndarray      # uint16 bf16 bits [T, H, 512]
    q_pe: np.ndarray
    kv_cache: np.ndarray    # uint16 or uint8 [P, 64, 576]
    page_table: np.ndarray  # int32 [B, max_pages]
    seq_lens: np.ndarray    # int32 [B]
    cu: np.ndarray          # int32 [B + 1]
    window: int
    sinks: int
    kv_dtype: str
    kv_scale: float
    scale: float


def make(new, total, heads, window=0, sinks=0, kv_dtype="bf16", seed=0, extra_q=0, extra_pages=3, q_gain=1.0,
         scale=SCALE):
    """One batch: request b brings new[b] tokens and has total[b] cached ones;
    extra_q query rows behind the last request."""
    rng = np.random.default_rng(seed)
    new, total = np.asarray(new, dtype=np.int64), np.asarray(total, dtype=np.int64)
    B = len(new)
    width = max(1, int(-(-total.max() // 64)))
    need = []
    for b in range(B):
        npg = int(-(-total[b] // 64))
        first = max(0, int(total[b] - new[b]) + 1 - window) if window else 0
        need.append([p for p in range(npg) if not window or p >= first // 64 or p * 64 < sinks])
    count = sum(len(x) for x in need) + extra_pages
    ids = rng.permutation(count).astype(np.int32)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, need[b]] = ids[at:at + len(need[b])]
        at += len(need[b])
    x = rng.standard_normal((count, 64, 576), dtype=np.float32)
    bits = W.f32_to_bf16_bits(x)
    kv_scale = 1.0
    if kv_dtype == "bf16":
        cache, nan = bits, W.BF16_NAN
    else:
        import torch

        kv_scale = float(np.float32(np.abs(x).max() / 448.0))
        cache = (torch.from_numpy(x) / kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
        nan = W.E4M3_NAN
    used = np.zeros((count, 64), dtype=bool)
    for b in range(B):
        for p in need[b]:
            used[table[b, p], :max(0, min(64, int(total[b]) - 64 * p))] = True
    cache[~used] = nan
    T = int(new.sum()) + extra_q
    qn = W.f32_to_bf16_bits(q_gain * rng.standard_normal((T, heads, 512), dtype=np.float32))
    qp = W.f32_to_bf16_bits(q_gain * rng.standard_normal((T, heads, 64), dtype=np.float32))
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return Chunk(qn, qp, cache, table, total.astype(np.int32), cu, window, sinks, kv_dtype, kv_scale, scale)


def to_cuda(a, kind="raw"):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a))
    if a.dtype == np.uint16:
        t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    return t.cuda()


def error_bounds(c, b, i):
    """Bounds on |out - exact| [H, 512] and |lse - exact| [H] of token i of
    request b, by counting roundings (bf16: half a step is 2^-8 relative; fp32
    arithmetic in tensor cores and registers: 2^-23 an operation).

    scores: 576 products summed in fp32, each partial sum at most
        S1 = sum |q||k| scale: 584 * 2^-23 * S1 (the scaling included); an
        e4m3 cache adds the part of q that hi + lo cannot hold, 2^-17 of the
        row's largest |q| per value;
    P: one bf16 rounding of every weight and a weight error of e^(2 d) - 1
        from scores and normaliser: (2^-8 + 2 d) sum softmax |v|;
    sums over n keys: n / 16 accumulations each way: (n / 16 + 64) 2^-23;
    out: one bf16 rounding, 2^-8 |out|.
    """
    import oracle

    pos = int(c.seq_lens[b]) - int(c.cu[b + 1] - c.cu[b]) + i
    keys = oracle.seen_keys(pos, c.window, c.sinks)
    rows = oracle.cache_rows_at(c.kv_cache, c.page_table[b], keys, c.kv_dtype, c.kv_scale)
    t = int(c.cu[b]) + i
    q = np.concatenate([oracle.bf16_bits_to_f64(c.q_nope[t]), oracle.bf16_bits_to_f64(c.q_pe[t])], axis=-1)
    s = (q @ rows.T) * c.scale
    w = np.exp(s - s.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    s1 = (np.abs(q) @ np.abs(rows).T).max(axis=1) * c.scale
    d = 584 * 2.0**-23 * s1
    if c.kv_dtype != "bf16":
        d = d + 2.0**-17 * np.abs(q).max(axis=1) * np.abs(rows).sum(axis=1).max() * c.scale
    n = len(keys)
    acc = (n / 16 + 64) * 2.0**-23
    ref = w @ rows[:, :512]
    mean_abs = w @ np.abs(rows[:, :512])
    out_tol = 2.0**-8 * np.abs(ref) + ((2.0**-8 + acc)[None] if np.ndim(acc) else 2.0**-8 + acc) * mean_abs
    out_tol = out_tol + (2 * d)[:, None] * mean_abs + 1e-30
    lse = s.max(axis=1) + np.log(np.exp(s - s.max(axis=1, keepdims=True)).sum(axis=1))
    lse_tol = d + acc + 8 * 2.0**-23 * (np.abs(lse) + 1)
    return out_tol, lse_tol
