"""The workloads on which the prompt, window, attention-mass and eviction
operators of the paged latent cache are measured.

A cached token is one latent row of 576 values, [c_kv (512) | k_pe (64)], in
64-token pages reached through a page table; an absorbed query row (q_nope
512 | q_pe 64) scores a row by their dot product times ``scale``.  The
operators:

* ``prefill``: attention of chunks of new tokens, of any lengths, over the
  paged cache (the new tokens' rows are in it already), causal, optionally
  over a sliding window plus a few first tokens;
* ``window``: the decode of one or a few new tokens per request over a
  sliding window plus a few first tokens;
* ``mass``: every cached token's accumulated attention weight, from the
  queries and log-sum-exps of a step;
* ``evict``: the tokens to keep by that weight, and the rows that move into
  the places of the dropped ones.
"""
import random

import numpy as np
import torch

own = False

PAGE = 64
LATENT = 512
ROW = 576
SCALE = 192.0 ** -0.5


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the last tokens of three short prompts: a call that latency bounds
        dict(name="prefill_tail", op="prefill", batch=3, heads=16, new_min=1, new_max=33, ctx_min=100, ctx_max=700,
             window=0, sinks=0, kv="bf16", lens=1),
        # two long prompts, 512 tokens a step, over 8K cached tokens: the bulk of prompt processing
        dict(name="prefill_chunk", op="prefill", batch=2, heads=128, new_min=512, new_max=512, ctx_min=8192,
             ctx_max=8192, window=0, sinks=0, kv="bf16", lens=2),
        # a mixed step of eight requests at different stages, 8-bit cache
        dict(name="prefill_ragged_e4m3", op="prefill", batch=8, heads=64, new_min=33, new_max=400, ctx_min=1000,
             ctx_max=16000, window=0, sinks=0, kv="e4m3", lens=3),
        # a long document read with a sliding window
        dict(name="prefill_window", op="prefill", batch=2, heads=128, new_min=700, new_max=1024, ctx_min=16000,
             ctx_max=16384, window=2048, sinks=4, kv="bf16", lens=4),
        # one request's next token
        dict(name="window_one", op="window", batch=1, heads=16, q_len=1, ctx_min=700, ctx_max=700, window=256,
             sinks=4, kv="bf16", lens=5),
        # a serving batch of long conversations
        dict(name="window_batch", op="window", batch=64, heads=64, q_len=1, ctx_min=4500, ctx_max=65536, window=4096,
             sinks=4, kv="bf16", lens=6),
        # two draft tokens per request, 8-bit cache, some contexts shorter than the window
        dict(name="window_drafts_e4m3", op="window", batch=128, heads=128, q_len=2, ctx_min=1000, ctx_max=16384,
             window=2048, sinks=16, kv="e4m3", lens=7),
        # the weights that a decode step gives the cached tokens
        dict(name="mass_step", op="mass", batch=64, heads=64, q_len=1, ctx_min=8192, ctx_max=8192, kv="bf16", lens=8),
        # the weights that a prompt's last 32 tokens give it, before its first eviction
        dict(name="mass_prompt_e4m3", op="mass", batch=4, heads=128, q_len=32, ctx_min=4000, ctx_max=32768, kv="e4m3",
             lens=9),
        # one short conversation back under its budget
        dict(name="evict_one", op="evict", batch=1, ctx_min=600, ctx_max=600, budget=512, sinks=4, recent=128,
             kv="bf16", lens=10),
        # a serving batch back under its budget after 64 to 128 more tokens each
        dict(name="evict_step", op="evict", batch=64, ctx_min=4160, ctx_max=4224, budget=4096, sinks=4, recent=512,
             kv="bf16", lens=11),
        # long prompts' first eviction
        dict(name="evict_prompt_e4m3", op="evict", batch=16, ctx_min=9000, ctx_max=32768, budget=4096, sinks=4,
             recent=1024, kv="e4m3", lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "window", "window", "mass", "evict"])
    kv = rng.choice(["bf16", "e4m3"])
    heads = rng.choice([16, 32, 64, 128, 20, 48])
    lens = rng.randrange(1 << 30)
    while True:
        if op == "prefill":
            hi = _log(rng, 1, 1024)
            ctx = _log(rng, 80, 20000)
            win = rng.random() < 0.4
            c = dict(op=op, batch=_log(rng, 1, 8), heads=heads, new_min=_log(rng, 1, hi), new_max=hi,
                     ctx_min=_log(rng, 64, ctx), ctx_max=ctx, window=_log(rng, 1, 8192) if win else 0,
                     sinks=rng.choice([0, 1, 4, 70]) if win else 0, kv=kv, lens=lens)
        elif op == "window":
            ctx = _log(rng, 80, 65536)
            c = dict(op=op, batch=_log(rng, 1, 128), heads=heads, q_len=rng.choice([1, 1, 2, 3]),
                     ctx_min=_log(rng, 64, ctx), ctx_max=ctx, window=_log(rng, 16, 8192),
                     sinks=rng.choice([0, 1, 4, 16, 100]), kv=kv, lens=lens)
        elif op == "mass":
            ctx = _log(rng, 80, 32768)
            c = dict(op=op, batch=_log(rng, 1, 64), heads=heads, q_len=rng.choice([1, 1, 2, 5, 32]),
                     ctx_min=_log(rng, 64, ctx), ctx_max=ctx, kv=kv, lens=lens)
        else:
            ctx = _log(rng, 100, 32768)
            budget = _log(rng, 64, 8192)
            recent = int(budget * rng.random() * 0.5)
            c = dict(op=op, batch=_log(rng, 1, 64), ctx_min=_log(rng, 64, ctx), ctx_max=ctx, budget=budget,
                     sinks=rng.choice([0, 1, 4, 16]), recent=recent, kv=kv, lens=lens)
        w = work(c)
        # no dearer than the largest listed case of its operator, in the plain form's memory too
        if w["flops"] <= {"prefill": 2.5e12, "window": 2.0e11, "mass": 7.0e11, "evict": 1}[op] and w["bytes"] <= 1.0e9:
            return c


def _lengths(c):
    """Per request: the new tokens of the step and the cached tokens in all."""
    r = random.Random(c["lens"])
    if c["op"] == "prefill":
        new = [r.randint(c["new_min"], c["new_max"]) for _ in range(c["batch"])]
        return new, [n + r.randint(c["ctx_min"], c["ctx_max"]) for n in new]
    return [c.get("q_len", 1)] * c["batch"], [r.randint(c["ctx_min"], c["ctx_max"]) for _ in range(c["batch"])]


def _seen(c, pos):
    """Keys that a query at position ``pos`` sees."""
    if not c.get("window"):
        return pos + 1
    lo = max(0, pos + 1 - c["window"])
    return pos + 1 - lo + min(c["sinks"], lo)


def _first(c, new, length):
    """The first key that the window of a request's first query holds."""
    return max(0, length - new + 1 - c["window"]) if c.get("window") else 0


def _moved(c, length):
    """Rows expected to move: those kept in the slots behind the budget."""
    k = c["budget"]
    if length <= k:
        return 0
    free = length - c["sinks"] - c["recent"]
    tail = max(0, length - k - c["recent"])
    return min(length - k, c["recent"]) + tail * (k - c["sinks"] - c["recent"]) / max(1, free)


def work(case):
    c = case
    row = ROW * (2 if c["kv"] == "bf16" else 1)
    new, total = _lengths(c)
    if c["op"] == "evict":
        by = sum(8 * n + 12 * min(n, c["budget"]) + 2 * row * _moved(c, n) for n in total)
        return {"bytes": by, "flops": 0}
    h = c["heads"]
    pairs = h * sum(sum(_seen(c, n - m + i) for i in range(m)) for m, n in zip(new, total))
    keys = sum(n - _first(c, m, n) + min(c.get("sinks", 0), _first(c, m, n)) for m, n in zip(new, total))
    rows = h * sum(new)
    if c["op"] == "mass":
        return {"bytes": rows * (2 * ROW + 4) + keys * (row + 8), "flops": 2.0 * ROW * pairs}
    return {"bytes": rows * (2 * ROW + 2 * LATENT + 4) + keys * row, "flops": 2.0 * (ROW + LATENT) * pairs}


# ------------------------------------------------------------------ inputs
def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _pool(c, new, total, gen):
    """A pool with a page for every 64 tokens that a query may see, handed out
    in random order; table entries of pages that the window has left are -1."""
    width = max(-(-n // PAGE) for n in total)
    col = torch.arange(width, device="cuda")[None]
    pages = torch.tensor([-(-n // PAGE) for n in total], device="cuda")[:, None]
    first = torch.tensor([_first(c, m, n) // PAGE for m, n in zip(new, total)], device="cuda")[:, None]
    used = (col < pages) & ((col >= first) | (col * PAGE < c.get("sinks", 0)))
    count = int(used.sum())
    table = torch.full((len(total), width), -1, dtype=torch.int32, device="cuda")
    table[used] = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    cache = torch.empty((count, PAGE, ROW), dtype=torch.bfloat16, device="cuda")
    for part in cache.split(2048):
        part.copy_(_normal(part.shape, gen))
    if c["kv"] == "bf16":
        return cache, 1.0, table
    kv_scale = float(cache.abs().max()) / 448.0
    codes = torch.empty(cache.shape, dtype=torch.uint8, device="cuda")
    for src, dst in zip(cache.split(2048), codes.split(2048)):
        dst.copy_((src.float() / kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    return codes, kv_scale, table


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    new, total = _lengths(c)
    s = {"c": c, "new": new, "total": total}
    s["cache"], s["kv_scale"], s["table"] = _pool(c, new, total, gen)
    s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    batch, cap = len(total), s["table"].shape[1] * PAGE
    if c["op"] == "evict":
        k = c["budget"]
        # heavy-tailed weights, a tenth of the tokens never attended to (equal, at zero)
        x = torch.randn((batch, cap), generator=gen, device="cuda")
        u = torch.rand((batch, cap), generator=gen, device="cuda")
        s["mass"] = torch.where(u < 0.1, torch.zeros_like(x), torch.exp(2.0 * x))
        # positions in the whole conversation: sinks first, the recent ones last, an earlier
        # eviction's order between them
        slot = torch.arange(cap, device="cuda")[None]
        mid = (slot >= c["sinks"]) & (slot < s["lens"][:, None] - c["recent"])
        key = torch.where(mid, c["sinks"] + u * (s["lens"][:, None] - c["recent"] - c["sinks"]), slot.float())
        s["positions"] = torch.argsort(torch.argsort(key, dim=1), dim=1).to(torch.int32)
        s["new_lens"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros((batch, k), dtype=torch.int32, device="cuda")
        s["mass_out"] = torch.zeros_like(s["mass"])
        s["positions_out"] = torch.zeros_like(s["positions"])
    else:
        h = c["heads"]
        shape = (sum(new), h) if c["op"] == "prefill" else (batch, new[0], h)
        s["q_nope"], s["q_pe"] = _normal(shape + (LATENT,), gen), _normal(shape + (64,), gen)
        if c["op"] == "mass":
            s["mass"] = torch.rand((batch, cap), generator=gen, device="cuda")
            s["mass_out"] = torch.zeros_like(s["mass"])
            rows, keep = _rows(s)
            s["lse"] = torch.logsumexp(_scores(s, rows, keep), dim=-1)
            del rows, keep
        else:
            s["out"] = torch.zeros(shape + (LATENT,), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.zeros(shape, dtype=torch.float32, device="cuda")
        if c["op"] == "prefill":
            s["starts"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    if own:
        import paged_mla_decode_09_gb300 as mla

        if c["op"] == "prefill":
            n = mla.mla_prefill_workspace_size(mla.make_prefill_dims(s["q_nope"], s["cache"], s["table"], s["lens"]))
        elif c["op"] == "window":
            n = mla.mla_decode_window_workspace_size(mla.make_dims(s["q_nope"], s["cache"], s["table"]))
        elif c["op"] == "mass":
            n = mla.mla_attn_mass_workspace_size(mla.make_dims(s["q_nope"], s["cache"], s["table"]))
        else:
            n = mla.mla_evict_workspace_size(batch, c["budget"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _values(s, codes):
    """Cache rows in 32 bits."""
    if s["c"]["kv"] == "bf16":
        return codes.float()
    return codes.view(torch.float8_e4m3fn).float() * s["kv_scale"]


def _take(s, table, at):
    """The rows at positions ``at`` [B, n] of the requests of ``table``."""
    page = torch.gather(table, 1, at // PAGE).long()
    return _values(s, s["cache"].view(-1, ROW)[page * PAGE + at % PAGE])


def _rows(s):
    """[B, longest, 576] rows and what each of the step's tokens sees of them."""
    n = s["lens"].long()[:, None]
    at = torch.arange(int(max(s["total"])), device="cuda")[None]
    rows = _take(s, s["table"], at.clamp(max=n - 1))
    q = s["q_nope"].shape[1]
    last = n - q + torch.arange(q, device="cuda")[None]
    return rows, at[:, None] <= last[:, :, None]


def _scores(s, rows, keep):
    """Scaled scores [B, q, heads, keys] in 32 bits, -inf where unseen."""
    q = torch.cat([s["q_nope"], s["q_pe"]], dim=-1).float()
    b, n, h, _ = q.shape
    sc = torch.matmul(q.view(b, n * h, ROW), rows.transpose(1, 2)).view(b, n, h, -1) * SCALE
    return sc.masked_fill_(~keep[:, :, None], float("-inf"))


def _attend(sc, rows):
    """Softmax over the last axis, and the latent part of the rows it weighs."""
    top = sc.amax(dim=-1, keepdim=True)
    w = torch.exp(sc - top)
    z = w.sum(dim=-1, keepdim=True)
    return torch.matmul(w, rows[..., :LATENT]) / z, (top + torch.log(z)).squeeze(-1)


def _plain_prefill(s):
    c, at = s["c"], 0
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        lo = _first(c, m, n)
        keys = torch.arange(lo, n, device="cuda")
        keys = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), keys])
        rows = _take(s, s["table"][b:b + 1], keys[None])[0]
        q = torch.cat([s["q_nope"][at:at + m], s["q_pe"][at:at + m]], dim=-1).float()
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        keep = keys[None] <= pos
        if c["window"]:
            keep &= (keys[None] > pos - c["window"]) | (keys[None] < c["sinks"])
        sc = (torch.matmul(q.view(-1, ROW), rows.T) * SCALE).view(m, c["heads"], -1)
        o, l = _attend(sc.masked_fill_(~keep[:, None], float("-inf")).view(m * c["heads"], -1), rows)
        s["out"][at:at + m] = o.view(m, c["heads"], LATENT).to(torch.bfloat16)
        s["lse"][at:at + m] = l.view(m, c["heads"])
        at += m
    return s["out"], s["lse"]


def _plain_window(s):
    c = s["c"]
    b, q, h, _ = s["q_nope"].shape
    n = s["lens"].long()[:, None]
    width = c["window"] + q - 1
    behind = n - width + torch.arange(width, device="cuda")[None]
    at = torch.cat([torch.arange(c["sinks"], device="cuda").expand(b, -1), behind], dim=1)
    once = torch.cat([at[:, :c["sinks"]] < n, behind >= c["sinks"]], dim=1)
    pos = (n - q + torch.arange(q, device="cuda")[None])[:, :, None]
    key = at[:, None]
    keep = once[:, None] & (key <= pos) & ((key > pos - c["window"]) | (key < c["sinks"]))
    rows = _take(s, s["table"], torch.where(once, at, n - 1))
    sc = _scores(s, rows, keep)
    o, l = _attend(sc.view(b, q * h, -1), rows)
    s["out"].copy_(o.view(b, q, h, LATENT))
    s["lse"].copy_(l.view(b, q, h))
    return s["out"], s["lse"]


def _plain_mass(s):
    rows, keep = _rows(s)
    w = torch.exp(_scores(s, rows, keep) - s["lse"][..., None])
    n = rows.shape[1]
    valid = torch.arange(n, device="cuda")[None] < s["lens"][:, None]
    s["mass_out"][:, :n] = torch.where(valid, s["mass"][:, :n] + w.sum(dim=(1, 2)), s["mass_out"][:, :n])
    return s["mass_out"]


def _plain_evict(s):
    c = s["c"]
    mass, pos, n = s["mass"], s["positions"], s["lens"].long()[:, None]
    slot = torch.arange(mass.shape[1], device="cuda")[None]
    valid = slot < n
    last = pos.masked_fill(~valid, -1).amax(dim=1, keepdim=True)
    firm = valid & ((pos < c["sinks"]) | (pos > last - c["recent"]))
    k = n.clamp(max=c["budget"])
    # the k tokens of the greatest weight, the firm ones before all, the lower slot before an equal one
    weight = mass.masked_fill(firm, float("inf")).masked_fill(~valid, float("-inf"))
    order = torch.sort(weight, dim=1, descending=True, stable=True).indices
    keep = torch.zeros_like(valid).scatter_(1, order, slot < k)
    holes = torch.nonzero((slot < k) & ~keep)
    moved = torch.nonzero((slot >= k) & keep)
    s["new_lens"].copy_(k[:, 0])
    kept = slot[:, :c["budget"]].masked_fill(slot[:, :c["budget"]] >= k, -1).to(torch.int32).contiguous()
    kept[holes[:, 0], holes[:, 1]] = moved[:, 1].to(torch.int32)
    s["kept"][:, :kept.shape[1]] = kept
    s["kept"][:, kept.shape[1]:] = -1
    have = kept >= 0
    old = kept.clamp(min=0).long()
    width = kept.shape[1]
    s["mass_out"][:, :width] = torch.where(have, torch.gather(mass, 1, old), s["mass_out"][:, :width])
    s["positions_out"][:, :width] = torch.where(have, torch.gather(pos, 1, old), s["positions_out"][:, :width])
    flat = s["cache"].view(-1, ROW)
    place = lambda at: s["table"][at[:, 0], at[:, 1] // PAGE].long() * PAGE + at[:, 1] % PAGE  # noqa: E731
    flat[place(holes)] = flat[place(moved)]
    return _evicted(s)


def _evicted(s):
    cache = s["cache"] if s["c"]["kv"] == "bf16" else s["cache"].view(torch.float8_e4m3fn)
    return s["new_lens"], s["kept"], s["mass_out"], s["positions_out"], cache


def run(state):
    s, c = state, state["c"]
    if own:
        import paged_mla_decode_09_gb300 as mla

        if c["op"] == "prefill":
            mla.mla_prefill(s["q_nope"], s["q_pe"], s["cache"], s["table"], s["lens"], s["starts"], c["window"],
                            c["sinks"], SCALE, s["kv_scale"], s["out"], s["lse"], s["workspace"])
            return s["out"], s["lse"]
        if c["op"] == "window":
            mla.mla_decode_window(s["q_nope"], s["q_pe"], s["cache"], s["table"], s["lens"], c["window"], c["sinks"],
                                  SCALE, s["kv_scale"], s["out"], s["lse"], s["workspace"])
            return s["out"], s["lse"]
        if c["op"] == "mass":
            mla.mla_attn_mass(s["q_nope"], s["q_pe"], s["cache"], s["table"], s["lens"], s["lse"], 0, SCALE,
                              s["kv_scale"], s["mass"], s["mass_out"], s["workspace"])
            return s["mass_out"]
        mla.mla_evict(s["mass"], s["positions"], s["lens"], s["table"], s["cache"], c["budget"], c["sinks"],
                      c["recent"], s["new_lens"], s["kept"], s["mass_out"], s["positions_out"], s["workspace"])
        return _evicted(s)
    return {"prefill": _plain_prefill, "window": _plain_window, "mass": _plain_mass, "evict": _plain_evict}[c["op"]](s)


# --------------------------------------------------------- 64-bit definition
def _exact_rows(s, b, n):
    """Request b's first n cache rows as 64-bit values (pages without an id: zeros)."""
    ids = s["table"][b, :-(-n // PAGE)].long()
    raw = s["cache"][ids.clamp(min=0)]
    if s["c"]["kv"] == "e4m3":
        raw = raw.view(torch.float8_e4m3fn)
    x = raw.to(torch.float64)
    if s["c"]["kv"] == "e4m3":
        x = x * s["kv_scale"]
    x[ids < 0] = 0.0
    return x.reshape(-1, ROW)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "evict":
        return _exact_evict(s)
    if c["op"] == "mass":
        result = s["mass_out"].to(torch.float64)
    else:
        result, lse = s["out"].to(torch.float64), s["lse"].to(torch.float64)
    at = 0
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        k = _exact_rows(s, b, n)
        part = slice(at, at + m) if c["op"] == "prefill" else b
        at += m
        qn, qp = s["q_nope"][part].to(torch.float64), s["q_pe"][part].to(torch.float64)
        t = torch.arange(n, device="cuda")
        total = torch.zeros(n, dtype=torch.float64, device="cuda")
        for i in range(m):  # one token at a time, over exactly the keys that it sees
            p = n - m + i
            seen = t[:p + 1]
            if c.get("window"):
                seen = seen[(seen > p - c["window"]) | (seen < c["sinks"])]
            kk = k[:p + 1] if len(seen) == p + 1 else k[seen]
            dot = (torch.einsum("hd,td->ht", qn[i], kk[:, :LATENT]) + torch.einsum("hd,td->ht", qp[i], kk[:, LATENT:])) * SCALE
            if c["op"] == "mass":
                total[:p + 1] += torch.exp(dot - s["lse"][b, i].to(torch.float64)[:, None]).sum(dim=0)
                continue
            l = torch.logsumexp(dot, dim=1)
            o = torch.exp(dot - l[:, None]) @ kk[:, :LATENT]
            if c["op"] == "prefill":
                result[at - m + i], lse[at - m + i] = o, l
            else:
                result[b, i], lse[b, i] = o, l
        if c["op"] == "mass":
            result[b, :n] = s["mass"][b, :n].to(torch.float64) + total
    return result if c["op"] == "mass" else (result, lse)


def _exact_evict(s):
    c = s["c"]
    mass, pos = s["mass"].double().cpu().numpy(), s["positions"].cpu().numpy()
    table = s["table"].cpu().numpy()
    new_lens, kept_all = np.zeros(len(s["total"]), np.int32), np.full((len(s["total"]), c["budget"]), -1, np.int32)
    mass_out, pos_out = np.zeros_like(mass), np.zeros_like(pos)
    cache = (s["cache"].view(torch.float8_e4m3fn) if c["kv"] == "e4m3" else s["cache"]).double()
    flat = cache.view(-1, ROW)
    src, dst = [], []
    for b, n in enumerate(s["total"]):
        k = min(n, c["budget"])
        last = int(pos[b, :n].max())
        firm = (pos[b, :n] < c["sinks"]) | (pos[b, :n] > last - c["recent"])
        ranked = sorted(range(n), key=lambda t: (0, 0.0, t) if firm[t] else (1, -mass[b, t], t))  # noqa: B023
        keep = set(ranked[:k])
        come = sorted(t for t in keep if t >= k)
        new_lens[b] = k
        for t in range(k):
            o = t if t in keep else come.pop(0)
            kept_all[b, t], mass_out[b, t], pos_out[b, t] = o, mass[b, o], pos[b, o]
            if o != t:
                src.append(int(table[b, o // PAGE]) * PAGE + o % PAGE)
                dst.append(int(table[b, t // PAGE]) * PAGE + t % PAGE)
    flat[torch.tensor(dst, dtype=torch.long, device="cuda")] = flat[torch.tensor(src, dtype=torch.long, device="cuda")]
    back = lambda a: torch.from_numpy(a).to("cuda")  # noqa: E731
    return back(new_lens), back(kept_all), back(mass_out), back(pos_out), cache
