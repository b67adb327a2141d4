"""The workloads on which the operators of a speculative step over the paged
latent cache are measured.

A cached token is one latent row of 576 values, [c_kv (512) | k_pe (64)], in
64-token pages reached through a page table.  A step brings every request a
few drafted tokens, the nodes of a tree: node i's parent comes before it (-1:
none), and the n nodes are the request's last n cached tokens.  The operators:

* ``rope``: rotary positions of a step's query and key parts, with the cache
  write of its rows;
* ``tree``: attention of the nodes, each over the tokens before the tree, its
  ancestors and itself;
* ``verify``: which nodes the target's probabilities accept, and the token
  that follows them, from given random numbers;
* ``commit``: the rows of the accepted nodes move together in every layer's
  cache;
* ``fork``: requests continue as several (a beam, samples of one prompt): full
  pages are shared, the started one is copied;
* ``resize``: pages are handed out and freed for the requests' new lengths.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
LATENT = 512
ROPE = 64
ROW = 576
SCALE = 192.0 ** -0.5


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one conversation with a small tree: a call that latency bounds
        dict(name="tree_one", op="tree", batch=1, heads=16, nodes_min=8, nodes_max=8, ctx_min=700, ctx_max=700,
             kv="bf16", lens=1),
        # a serving batch, large trees, 8-bit cache
        dict(name="tree_batch_e4m3", op="tree", batch=16, heads=128, nodes_min=20, nodes_max=48, ctx_min=1500,
             ctx_max=9000, kv="e4m3", lens=2),
        # one request, a chain of four drafts sampled from the drafter
        dict(name="verify_one", op="verify", batch=1, nodes_min=5, nodes_max=5, vocab=32000, draft=True, chain=True,
             lens=3),
        # a serving batch of chains
        dict(name="verify_chains", op="verify", batch=64, nodes_min=6, nodes_max=6, vocab=131072, draft=True,
             chain=True, lens=4),
        # the tokens of one request's next step
        dict(name="rope_one", op="rope", batch=1, heads=16, new_min=4, new_max=4, ctx_min=900, ctx_max=900, rotary=64,
             interleaved=True, factor=1.0, original=0, kv="bf16", depths=True, lens=5),
        # prompt chunks far inside a long context, 8-bit cache
        dict(name="rope_prompt_e4m3", op="rope", batch=4, heads=128, new_min=1000, new_max=2048, ctx_min=60000,
             ctx_max=150000, rotary=64, interleaved=False, factor=40.0, original=4096, kv="e4m3", depths=False,
             lens=6),
        # one request's accepted nodes, a few layers
        dict(name="commit_one", op="commit", batch=1, layers=4, nodes_min=8, nodes_max=8, ctx_min=700, ctx_max=700,
             kv="bf16", lens=7),
        # a serving batch's, a deep model
        dict(name="commit_batch", op="commit", batch=64, layers=24, nodes_min=12, nodes_max=32, ctx_min=300,
             ctx_max=8000, kv="bf16", lens=8),
        # four samples of one prompt
        dict(name="fork_samples", op="fork", sources=1, children=4, layers=8, ctx_min=1000, ctx_max=1000, kv="bf16",
             lens=9),
        # a beam step of many requests, 8-bit cache
        dict(name="fork_beams_e4m3", op="fork", sources=64, children=64, layers=16, ctx_min=200, ctx_max=1600,
             kv="e4m3", lens=10),
        # a small server's step
        dict(name="resize_few", op="resize", batch=4, columns=32, pages=512, lens=11),
        # a large one's
        dict(name="resize_many", op="resize", batch=256, columns=512, pages=131072, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "verify", "rope", "commit", "fork", "resize"])
    kv = rng.choice(["bf16", "e4m3"])
    heads = rng.choice([16, 32, 64, 128, 20, 48])
    lens = rng.randrange(1 << 30)
    while True:
        if op == "tree":
            hi, ctx = _log(rng, 1, 200), _log(rng, 1, 32768)
            c = dict(op=op, batch=_log(rng, 1, 64), heads=heads, nodes_min=_log(rng, 1, hi), nodes_max=hi,
                     ctx_min=_log(rng, 1, ctx), ctx_max=ctx, kv=kv, lens=lens)
        elif op == "verify":
            hi = _log(rng, 1, 64)
            c = dict(op=op, batch=_log(rng, 1, 128), nodes_min=_log(rng, 1, hi), nodes_max=hi,
                     vocab=_log(rng, 1000, 200000), draft=rng.random() < 0.6, chain=rng.random() < 0.5, lens=lens)
        elif op == "rope":
            hi, ctx = _log(rng, 1, 2048), _log(rng, 1, 160000)
            factor = rng.choice([1.0, 1.0, 4.0, 40.0])
            c = dict(op=op, batch=_log(rng, 1, 64), heads=heads, new_min=_log(rng, 1, hi), new_max=hi,
                     ctx_min=_log(rng, 1, ctx), ctx_max=ctx, rotary=rng.choice([64, 64, 32, 16, 48]),
                     interleaved=rng.random() < 0.5, factor=factor,
                     original=rng.choice([0, 4096]) if factor > 1 else 0, kv=kv, depths=rng.random() < 0.5, lens=lens)
        elif op == "commit":
            hi, ctx = _log(rng, 1, 64), _log(rng, 1, 16000)
            c = dict(op=op, batch=_log(rng, 1, 128), layers=_log(rng, 1, 64), nodes_min=_log(rng, 1, hi), nodes_max=hi,
                     ctx_min=_log(rng, 1, ctx), ctx_max=ctx, kv=kv, lens=lens)
        elif op == "fork":
            ctx = _log(rng, 1, 8000)
            n = _log(rng, 1, 64)
            c = dict(op=op, sources=n, children=_log(rng, 1, 128), layers=_log(rng, 1, 32), ctx_min=_log(rng, 1, ctx),
                     ctx_max=ctx, kv=kv, lens=lens)
        else:
            cols = _log(rng, 4, 512)
            batch = _log(rng, 1, 256)
            c = dict(op=op, batch=batch, columns=cols, pages=max(batch * cols, _log(rng, 64, 131072)), lens=lens)
        w = work(c)
        # no dearer than the largest listed case of its operator, in the inputs' memory too
        if (w["flops"] <= {"tree": 1.2e12}.get(op, 1e9) and _memory(c) <= 6e8
                and w["bytes"] <= {"tree": 1e9, "verify": 7e7, "rope": 2.6e8}.get(op, 5e7)):
            return c


def _lengths(c):
    """Per request: the step's new tokens and the cached tokens in all."""
    r = random.Random(c["lens"])
    lo, hi = (c["new_min"], c["new_max"]) if c["op"] == "rope" else (c["nodes_min"], c["nodes_max"])
    new = [r.randint(lo, hi) for _ in range(c["batch"])]
    if c["op"] == "verify":
        return new, new
    return new, [n + r.randint(c["ctx_min"], c["ctx_max"]) for n in new]


def _trees(c, new):
    """Per request its nodes' parents: a root, then nodes that mostly hang on
    one of the few before them."""
    r = random.Random(c["lens"] + 1)
    if c.get("chain"):
        return [[i - 1 for i in range(n)] for n in new]
    return [[-1] + [r.randint(max(0, i - 6), i - 1) for i in range(1, n)] for n in new]


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _paths(c, trees):
    """Per request the nodes accepted: the root and some of a line below it."""
    r = random.Random(c["lens"] + 2)
    paths = []
    for parents in trees:
        at, path = 0, [0]
        while r.random() < 0.75:
            below = [j for j, q in enumerate(parents) if q == at]
            if not below:
                break
            at = r.choice(below)
            path.append(at)
        paths.append(path)
    return paths


def _forks(c):
    """Lengths of the sources, and every child's source."""
    r = random.Random(c["lens"])
    lens = [r.randint(c["ctx_min"], c["ctx_max"]) for _ in range(c["sources"])]
    return lens, [r.randrange(c["sources"]) for _ in range(c["children"])]


def _row(c):
    return ROW * (2 if c["kv"] == "bf16" else 1)


def _memory(c):
    """Bytes of the largest inputs."""
    if c["op"] == "verify":
        return 4 * c["vocab"] * sum(_lengths(c)[0])
    if c["op"] == "fork":
        lens, src = _forks(c)
        return c["layers"] * PAGE * _row(c) * (sum(-(-n // PAGE) for n in lens) + len(src) + 4)
    if c["op"] == "commit":
        return c["layers"] * PAGE * _row(c) * c["batch"] * (2 + c["nodes_max"] // PAGE)
    return 0


def work(case):
    c = case
    if c["op"] == "resize":
        # tables and counts, once in and once out
        return {"bytes": 8 * (c["batch"] * c["columns"] + c["pages"]), "flops": 0}
    if c["op"] == "fork":
        lens, src = _forks(c)
        width = max(-(-n // PAGE) for n in lens)
        pages = sum(-(-n // PAGE) for n in lens) + len(src)
        tails = sum(lens[s] % PAGE for s in src)
        return {"bytes": 2 * tails * _row(c) * c["layers"] + 8 * (len(src) * width + pages), "flops": 0}
    new, total = _lengths(c)
    if c["op"] == "verify":
        # of every request one row is sampled from (all its entries add up), with the draft's beside it where a
        # draft was rejected, which ends most requests
        rows = c["batch"] * (2 if c["draft"] and c["nodes_max"] > 1 else 1)
        return {"bytes": 4 * c["vocab"] * rows, "flops": 0}
    if c["op"] == "rope":
        t = sum(new)
        return {"bytes": t * (c["heads"] * ROPE * 4 + 2 * ROW + _row(c)), "flops": 3.0 * t * (c["heads"] + 1) * c["rotary"]}
    trees = _trees(c, new)
    if c["op"] == "commit":
        moved = sum(sum(k != j for k, j in enumerate(p)) for p in _paths(c, trees))
        return {"bytes": 2 * moved * _row(c) * c["layers"] + 4 * sum(map(len, trees)), "flops": 0}
    h = c["heads"]
    pairs = h * sum(m * (n - m) + m + sum(_depths(t)) for m, n, t in zip(new, total, trees))
    rows = h * sum(new)
    return {"bytes": rows * (2 * ROW + 2 * LATENT + 4) + sum(total) * _row(c), "flops": 2.0 * (ROW + LATENT) * pairs}


# ------------------------------------------------------------------ inputs
def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(counts):
    return _i32([0] + np.cumsum(counts).tolist())


def _rows_of(c, shape, gen):
    """A cache of the given shape [..., 576], and its scale."""
    cache = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = cache.view(-1, ROW)
    for part in flat.split(1 << 17):
        part.copy_(_normal(part.shape, gen))
    if c["kv"] == "bf16":
        return cache, 1.0
    kv_scale = float(flat.abs().max()) / 448.0
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for src, dst in zip(flat.split(1 << 17), codes.view(-1, ROW).split(1 << 17)):
        dst.copy_((src.float() / kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    return codes, kv_scale


def _table(total, first, gen):
    """A page for every 64 tokens from token first[b] on, in random order; the
    entries before them are -1."""
    width = max(1, max(-(-n // PAGE) for n in total))
    col = torch.arange(width, device="cuda")[None]
    last = torch.tensor([-(-n // PAGE) for n in total], device="cuda")[:, None]
    used = (col < last) & (col >= torch.tensor([f // PAGE for f in first], device="cuda")[:, None])
    count = int(used.sum())
    table = torch.full((len(total), width), -1, dtype=torch.int32, device="cuda")
    table[used] = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    return table, max(1, count)


def frequencies(c):
    """Radians a token of every rotated pair: 10000^(-2 i / R), divided by the
    factor where a pair turns rarely within the original length."""
    out = []
    for i in range(c["rotary"] // 2):
        f = 10000.0 ** (-2.0 * i / c["rotary"])
        turns = c["original"] * f / (2.0 * math.pi)
        keep = 0.0 if not c["original"] else min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
        out.append(f if c["factor"] == 1.0 else keep * f + (1.0 - keep) * f / c["factor"])
    return out


def _amplitude(c):
    return 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"c": c}
    {"tree": _prepare_tree, "verify": _prepare_verify, "rope": _prepare_rope, "commit": _prepare_commit,
     "fork": _prepare_fork, "resize": _prepare_resize}[c["op"]](s, c, gen)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _prepare_tree(s, c, gen):
    s["new"], s["total"] = _lengths(c)
    s["table"], count = _table(s["total"], [0] * c["batch"], gen)
    s["cache"], s["kv_scale"] = _rows_of(c, (count, PAGE, ROW), gen)
    s["lens"], s["starts"] = _i32(s["total"]), _offsets(s["new"])
    s["parents"] = _i32(sum(_trees(c, s["new"]), []))
    shape = (sum(s["new"]), c["heads"])
    s["q_nope"], s["q_pe"] = _normal(shape + (LATENT,), gen), _normal(shape + (ROPE,), gen)
    s["out"] = torch.zeros(shape + (LATENT,), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(shape, dtype=torch.float32, device="cuda")
    if own:
        import paged_mla_decode_09_gb300 as mla

        dims = mla.make_prefill_dims(s["q_nope"], s["cache"], s["table"], s["lens"])
        s["workspace"] = torch.empty(mla.mla_decode_tree_workspace_size(dims), dtype=torch.uint8, device="cuda")


def _prepare_verify(s, c, gen):
    s["new"], _ = _lengths(c)
    trees = _trees(c, s["new"])
    v, count = c["vocab"], sum(s["new"])
    s["starts"], s["parents"] = _offsets(s["new"]), _i32(sum(trees, []))
    s["p"] = torch.empty((count, v), device="cuda")
    draft = torch.empty((count, v), device="cuda")
    for a in range(0, count, 64):  # a drafter that is mostly near the target
        x = 5.0 * torch.randn((min(64, count - a), v), generator=gen, device="cuda")
        s["p"][a:a + 64] = torch.softmax(x, dim=1)
        draft[a:a + 64] = torch.softmax(x + 0.8 * torch.randn(x.shape, generator=gen, device="cuda"), dim=1)
    # a child's token: a draw of its parent's draft distribution, or the best ones of it in turn
    at = [b + max(q, 0) for b, t in zip(np.cumsum([0] + s["new"]).tolist(), trees) for q in t]
    at = torch.tensor(at, device="cuda")
    if c["draft"]:
        s["q"] = draft
        tok = torch.cat([torch.multinomial(draft[i], 1, generator=gen)[:, 0] for i in at.split(64)])
    else:
        s["q"] = None
        nth = [sum(q == t[j] for q in t[:j]) for t in trees for j in range(len(t))]
        best = torch.cat([torch.topk(draft[i], min(v, max(nth) + 1), dim=1).indices for i in at.split(64)])
        tok = best.gather(1, torch.tensor(nth, device="cuda")[:, None])[:, 0]
    s["tokens"] = tok.to(torch.int32)
    s["accept"] = torch.rand(count, generator=gen, device="cuda")
    s["sample"] = torch.rand(c["batch"], generator=gen, device="cuda")
    shape = (c["batch"], c["nodes_max"])
    s["path"], s["next"] = (torch.zeros(shape, dtype=torch.int32, device="cuda") for _ in range(2))
    s["count"] = torch.zeros(c["batch"], dtype=torch.int32, device="cuda")


def _prepare_rope(s, c, gen):
    s["new"], s["total"] = _lengths(c)
    first = [n - m for m, n in zip(s["new"], s["total"])]
    s["table"], count = _table(s["total"], first, gen)
    s["cache"], _ = _rows_of(c, (count, PAGE, ROW), gen)
    t = sum(s["new"])
    s["rows"] = _normal((t, ROW), gen)
    s["kv_scale"] = 1.0 if c["kv"] == "bf16" else 1.5 * float(s["rows"].abs().max()) / 448.0
    s["q_pe"] = _normal((t, c["heads"], ROPE), gen)
    s["q_out"] = torch.zeros_like(s["q_pe"])
    s["lens"], s["starts"] = _i32(s["total"]), _offsets(s["new"])
    at = [list(range(m)) for m in s["new"]]
    if c["depths"]:  # drafted trees: nodes of one depth share a position
        at = [_depths(t) for t in _trees(c, s["new"])]
    s["positions"] = _i32([f + x for f, d in zip(first, at) for x in d])
    if own:
        import paged_mla_decode_09_gb300 as mla

        s["plan"] = mla.mla_rope_plan(c["rotary"], base=10000.0, factor=c["factor"], original_len=c["original"],
                                      fast=32.0, slow=1.0, interleaved=c["interleaved"], amplitude=_amplitude(c))
    s["freq"] = torch.tensor(frequencies(c), dtype=torch.float64, device="cuda")


def _prepare_commit(s, c, gen):
    s["new"], s["total"] = _lengths(c)
    s["table"], count = _table(s["total"], [n - m for m, n in zip(s["new"], s["total"])], gen)
    s["cache"], _ = _rows_of(c, (c["layers"], count, PAGE, ROW), gen)
    s["lens"], s["starts"] = _i32(s["total"]), _offsets(s["new"])
    paths = _paths(c, _trees(c, s["new"]))
    s["path"] = _i32([p + [-1] * (c["nodes_max"] - len(p)) for p in paths])
    s["count"] = _i32([len(p) for p in paths])
    s["new_lens"] = torch.zeros(c["batch"], dtype=torch.int32, device="cuda")


def _prepare_fork(s, c, gen):
    s["total"], src = _forks(c)
    table, count = _table(s["total"], [0] * c["sources"], gen)
    pool = count + c["children"] + 3
    ids = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    s["table"] = torch.where(table >= 0, ids[table.clamp(min=0).long()], table)
    s["refs"] = torch.zeros(pool, dtype=torch.int32, device="cuda")
    s["refs"][s["table"][s["table"] >= 0].long()] = 1
    s["cache"], _ = _rows_of(c, (c["layers"], pool, PAGE, ROW), gen)
    s["lens"], s["src"] = _i32(s["total"]), _i32(src)
    s["table_out"] = torch.zeros((c["children"], s["table"].shape[1]), dtype=torch.int32, device="cuda")
    s["refs_out"] = torch.zeros_like(s["refs"])
    if own:
        import paged_mla_decode_09_gb300 as mla

        n = mla.mla_page_fork_workspace_size(c["sources"], c["children"], s["table"].shape[1], pool)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")


def _prepare_resize(s, c, gen):
    r = random.Random(c["lens"])
    cap = c["columns"] * PAGE
    old = [_log(r, 1, cap) for _ in range(c["batch"])]
    # most requests grow by a few tokens; some have ended, some lose drafts, some receive a prompt chunk
    new = []
    for n in old:
        k = r.random()
        new.append(min(cap, n + r.randint(1, 8) if k < 0.7 else 0 if k < 0.8 else max(0, n - r.randint(1, 64))
                       if k < 0.9 else n + r.randint(100, 2048)))
    have = [-(-n // PAGE) for n in old]
    ids = torch.randperm(c["pages"], generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(c["columns"], device="cuda")[None]
    used = col < torch.tensor(have, device="cuda")[:, None]
    table = torch.full((c["batch"], c["columns"]), -1, dtype=torch.int32, device="cuda")
    table[used] = ids[:int(used.sum())]
    # every other request shares the beginning of the one before it
    for b in range(1, c["batch"], 2):
        n = min(have[b], have[b - 1]) // 2
        table[b, :n] = table[b - 1, :n]
    s["table"] = table
    s["refs"] = torch.bincount(table[table >= 0].long(), minlength=c["pages"]).to(torch.int32)
    s["lens"] = _i32(new)
    s["table_out"], s["refs_out"] = torch.zeros_like(s["table"]), torch.zeros_like(s["refs"])
    if own:
        import paged_mla_decode_09_gb300 as mla

        n = mla.mla_page_resize_workspace_size(c["batch"], c["columns"], c["pages"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------- plain forms
def _cache_values(s):
    return s["cache"] if s["c"]["kv"] == "bf16" else s["cache"].view(torch.float8_e4m3fn)


def _ancestors(s):
    """[T, most nodes] truth: the node and its ancestors, by place in the tree."""
    parents, starts = s["parents"].long(), s["starts"].long()
    t = torch.arange(parents.shape[0], device="cuda")
    start = starts[torch.searchsorted(starts, t, right=True) - 1]
    at, live = t - start, torch.ones_like(t, dtype=torch.bool)
    most = max(s["new"])
    seen = torch.zeros((t.shape[0], most), dtype=torch.bool, device="cuda")
    for _ in range(most):
        seen |= live[:, None] & (torch.arange(most, device="cuda")[None] == at[:, None])
        up = parents[start + at]
        live &= up >= 0
        at = up.clamp(min=0)
    return seen


def _plain_tree(s):
    c, at, seen = s["c"], 0, _ancestors(s)
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        pages = s["table"][b, :-(-n // PAGE)].long()
        rows = _cache_values({"c": c, "cache": s["cache"][pages]}).float().view(-1, ROW)[:n]
        if c["kv"] == "e4m3":
            rows = rows * s["kv_scale"]
        q = torch.cat([s["q_nope"][at:at + m], s["q_pe"][at:at + m]], dim=-1).float()
        keep = torch.ones((m, n), dtype=torch.bool, device="cuda")
        keep[:, n - m:] = seen[at:at + m, :m]
        sc = (torch.matmul(q.view(-1, ROW), rows.T) * SCALE).view(m, c["heads"], n)
        sc = sc.masked_fill_(~keep[:, None], float("-inf"))
        top = sc.amax(dim=-1, keepdim=True)
        w = torch.exp(sc - top)
        z = w.sum(dim=-1, keepdim=True)
        s["out"][at:at + m] = (torch.matmul(w, rows[:, :LATENT]) / z).to(torch.bfloat16)
        s["lse"][at:at + m] = (top + torch.log(z)).squeeze(-1)
        at += m
    return s["out"], s["lse"]


def _plain_verify(s):
    c, p, q = s["c"], s["p"], s["q"]
    start, end = s["starts"][:-1].long(), s["starts"][1:].long()
    parents, tokens = s["parents"].long(), s["tokens"].long()
    b = torch.arange(c["batch"], device="cuda")
    cur, count = torch.zeros_like(start), torch.ones_like(start)
    w, z = p[start].double(), torch.ones(c["batch"], dtype=torch.float64, device="cuda")
    s["path"].fill_(-1)
    s["next"].fill_(-1)
    s["path"][:, 0] = 0
    cols = s["path"].shape[1]
    for j in range(1, max(s["new"])):
        at = (start + j).clamp(max=parents.shape[0] - 1)
        live = (start + j < end) & (parents[at] == cur) & (count < cols)
        x = tokens[at]
        wx = w[b, x]
        qx = q[start + cur, x].double() if q is not None else torch.ones_like(wx)
        yes = live & (s["accept"][at].double() * z * qx < wx)
        no = live & ~yes
        if q is not None:
            rest = (w - z[:, None] * q[start + cur].double()).clamp(min=0)
            left = rest.sum(dim=1)
        else:
            rest = w.scatter(1, x[:, None], 0.0)
            left = (z - wx).clamp(min=0)
        w = torch.where(yes[:, None], p[at].double(), torch.where(no[:, None], rest, w))
        z = torch.where(yes, torch.ones_like(z), torch.where(no, left, z))
        put = count.clamp(max=cols - 1)
        s["path"][b, put] = torch.where(yes, j, s["path"][b, put].long()).to(torch.int32)
        s["next"][b, count - 1] = torch.where(yes, x, s["next"][b, count - 1].long()).to(torch.int32)
        cur = torch.where(yes, j, cur)
        count = count + yes
    total = w.sum(dim=1)
    w = torch.where((total > 0)[:, None], w, p[start + cur].double())
    total = w.sum(dim=1)
    below = torch.cumsum(w, dim=1) <= (s["sample"].double() * total)[:, None]
    s["next"][b, count - 1] = below.sum(dim=1).clamp(max=c["vocab"] - 1).to(torch.int32)
    s["count"].copy_(count)
    return s["path"], s["next"], s["count"]


def _turned(s, x):
    """x [T, n, 64] in 32 bits with its first ``rotary`` values rotated."""
    c = s["c"]
    r = c["rotary"]
    angle = s["positions"].double()[:, None] * s["freq"][None]
    co = (torch.cos(angle) * _amplitude(c)).float()[:, None]
    si = (torch.sin(angle) * _amplitude(c)).float()[:, None]
    out = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
    if c["interleaved"]:
        out[..., 0:r:2], out[..., 1:r:2] = a * co - b * si, a * si + b * co
    else:
        out[..., :r // 2], out[..., r // 2:r] = a * co - b * si, a * si + b * co
    return out


def _slots(s):
    """The cache row of every new token of the step."""
    starts = s["starts"].long()
    t = torch.arange(s["positions"].shape[0], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    at = s["lens"].long()[b] - starts[b + 1] + t
    return s["table"][b, at // PAGE].long() * PAGE + at % PAGE


def _plain_rope(s):
    s["q_out"].copy_(_turned(s, s["q_pe"].float()))
    rows = s["rows"].float()
    rows[:, LATENT:] = _turned(s, rows[:, None, LATENT:])[:, 0]
    flat = _cache_values(s).view(-1, ROW)
    if s["c"]["kv"] == "e4m3":
        codes = (rows / s["kv_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        flat.view(torch.uint8)[_slots(s)] = codes.view(torch.uint8)
    else:
        flat[_slots(s)] = rows.to(torch.bfloat16)
    return s["q_out"], _cache_values(s)


def _plain_commit(s):
    k = torch.arange(s["path"].shape[1], device="cuda")[None]
    base = (s["lens"] - (s["starts"][1:] - s["starts"][:-1])).long()[:, None]
    use = (k < s["count"][:, None]) & (s["path"] != k)
    b, k = torch.nonzero(use, as_tuple=True)
    frm, to = base[b, 0] + s["path"][b, k].long(), base[b, 0] + k
    flat = s["cache"].view(s["cache"].shape[0], -1, ROW)
    place = lambda at: s["table"][b, at // PAGE].long() * PAGE + at % PAGE  # noqa: E731
    flat[:, place(to)] = flat[:, place(frm)]
    s["new_lens"].copy_(base[:, 0] + s["count"])
    return s["new_lens"], _cache_values(s)


def _plain_fork(s):
    src, n = s["src"].long(), s["lens"].long()
    s["table_out"].copy_(s["table"][src])
    full, tail = n[src] // PAGE, n[src] % PAGE
    col = torch.arange(s["table"].shape[1], device="cuda")[None]
    shared = s["table_out"][col < full[:, None]].long()
    s["refs_out"].copy_(s["refs"])
    s["refs_out"].index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    free = torch.nonzero(s["refs_out"] == 0)[:, 0]
    child = torch.nonzero(tail > 0)[:, 0]
    page = free[:child.shape[0]]
    s["refs_out"][page] = 1
    s["table_out"][child, full[child]] = page.to(torch.int32)
    s["table_out"][col >= (full + (tail > 0))[:, None]] = -1
    old = s["table"][src[child], full[child]].long()
    keep = torch.arange(PAGE, device="cuda")[None] < tail[child][:, None]
    i, j = torch.nonzero(keep, as_tuple=True)
    flat = s["cache"].view(s["cache"].shape[0], -1, ROW)
    flat[:, page[i] * PAGE + j] = flat[:, old[i] * PAGE + j]
    return s["table_out"], s["refs_out"], _cache_values(s)


def _plain_resize(s):
    table, need = s["table"], (s["lens"].long() + PAGE - 1) // PAGE
    want = torch.arange(table.shape[1], device="cuda")[None] < need[:, None]
    back = table[(table >= 0) & ~want].long()
    s["refs_out"].copy_(s["refs"])
    s["refs_out"].index_add_(0, back, torch.full_like(back, -1, dtype=torch.int32))
    free = torch.nonzero(s["refs_out"] == 0)[:, 0]
    s["table_out"].copy_(table.masked_fill(~want, -1))
    empty = torch.nonzero(want & (table < 0))
    page = free[:empty.shape[0]]
    s["table_out"][empty[:, 0], empty[:, 1]] = page.to(torch.int32)
    s["refs_out"][page] = 1
    return s["table_out"], s["refs_out"]


def run(state):
    s, c = state, state["c"]
    if not own:
        return {"tree": _plain_tree, "verify": _plain_verify, "rope": _plain_rope, "commit": _plain_commit,
                "fork": _plain_fork, "resize": _plain_resize}[c["op"]](s)
    import paged_mla_decode_09_gb300 as mla

    if c["op"] == "tree":
        mla.mla_decode_tree(s["q_nope"], s["q_pe"], s["cache"], s["table"], s["lens"], s["starts"], s["parents"],
                            SCALE, s["kv_scale"], s["out"], s["lse"], s["workspace"])
        return s["out"], s["lse"]
    if c["op"] == "verify":
        mla.mla_verify(s["p"], s["q"], s["tokens"], s["parents"], s["starts"], s["accept"], s["sample"], s["path"],
                       s["next"], s["count"], s["status"])
        return s["path"], s["next"], s["count"]
    if c["op"] == "rope":
        mla.mla_rope_pack(s["plan"], s["q_pe"], s["rows"], s["positions"], s["table"], s["lens"], s["starts"],
                          s["kv_scale"], s["q_out"], s["cache"], s["status"])
        return s["q_out"], _cache_values(s)
    if c["op"] == "commit":
        mla.mla_tree_commit(s["cache"], s["table"], s["lens"], s["starts"], s["path"], s["count"], s["new_lens"],
                            s["status"])
        return s["new_lens"], _cache_values(s)
    if c["op"] == "fork":
        mla.mla_page_fork(s["src"], s["lens"], s["table"], s["refs"], s["cache"], s["table_out"], s["refs_out"],
                          s["workspace"])
        return s["table_out"], s["refs_out"], _cache_values(s)
    mla.mla_page_resize(s["lens"], s["table"], s["refs"], s["table_out"], s["refs_out"], s["workspace"])
    return s["table_out"], s["refs_out"]


# --------------------------------------------------------- 64-bit definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "rope": _exact_rope, "commit": _exact_commit,
            "fork": _exact_fork, "resize": _exact_resize}[s["c"]["op"]](s)


def _doubles(s):
    return _cache_values(s).to(torch.float64)


def _exact_tree(s):
    c = s["c"]
    out, lse = s["out"].to(torch.float64), s["lse"].to(torch.float64)
    parents, at = s["parents"].tolist(), 0
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        raw = s["cache"][s["table"][b, :-(-n // PAGE)].long()]
        k = _doubles({"c": c, "cache": raw}).reshape(-1, ROW)[:n]
        k = k * s["kv_scale"] if c["kv"] == "e4m3" else k
        before = torch.arange(n - m, device="cuda")
        for i in range(m):  # one node at a time, over exactly the keys that it sees
            line, j = [], i
            while j >= 0:
                line.append(n - m + j)
                j = parents[at + j]
            kk = k[torch.cat([before, torch.tensor(line, device="cuda")])]
            q = torch.cat([s["q_nope"][at + i], s["q_pe"][at + i]], dim=1).to(torch.float64)
            dot = q @ kk.T * SCALE
            lse[at + i] = torch.logsumexp(dot, dim=1)
            out[at + i] = torch.exp(dot - lse[at + i][:, None]) @ kk[:, :LATENT]
        at += m
    return out, lse


def _exact_verify(s):
    c = s["c"]
    path = np.full(s["path"].shape, -1, np.int32)
    nxt = np.full(s["next"].shape, -1, np.int32)
    count = np.zeros(c["batch"], np.int32)
    parents, tokens = s["parents"].tolist(), s["tokens"].tolist()
    accept, sample = s["accept"].tolist(), s["sample"].tolist()
    row = lambda x, i: x[i].cpu().numpy().astype(np.float64)  # noqa: E731
    t0 = 0
    for b, n in enumerate(s["new"]):
        line, weight, mass, last = [0], row(s["p"], t0), 1.0, 0
        while True:
            child = next((j for j in range(last + 1, n) if parents[t0 + j] == line[-1]), None)
            if child is None or len(line) == path.shape[1]:
                break
            last, x = child, tokens[t0 + child]
            drafted = row(s["q"], t0 + line[-1]) if s["q"] is not None else None
            if accept[t0 + child] * mass * (1.0 if drafted is None else drafted[x]) < weight[x]:
                nxt[b, len(line) - 1] = x
                line.append(child)
                weight, mass = row(s["p"], t0 + child), 1.0
            elif drafted is None:
                mass = max(0.0, mass - weight[x])
                weight[x] = 0.0
            else:
                weight = np.maximum(0.0, weight - mass * drafted)
                mass = math.fsum(weight)
        if not weight.sum() > 0:
            weight = row(s["p"], t0 + line[-1])
        sums = np.cumsum(weight)
        nxt[b, len(line) - 1] = min(c["vocab"] - 1, int(np.searchsorted(sums, sample[b] * sums[-1], side="right")))
        path[b, :len(line)] = line
        count[b] = len(line)
        t0 += n
    return tuple(torch.from_numpy(a).to("cuda") for a in (path, nxt, count))


def _exact_rope(s):
    c = s["c"]
    half = c["rotary"] // 2
    co, si = [], []
    for p in s["positions"].tolist():
        co.append([math.cos(p * f) * _amplitude(c) for f in frequencies(c)])
        si.append([math.sin(p * f) * _amplitude(c) for f in frequencies(c)])
    co, si = (torch.tensor(a, dtype=torch.float64, device="cuda") for a in (co, si))

    def turn(x):  # [..., T, 64]
        x = x.to(torch.float64)
        y = x.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, half + i)
            y[..., a] = x[..., a] * co[:, i] - x[..., b] * si[:, i]
            y[..., b] = x[..., a] * si[:, i] + x[..., b] * co[:, i]
        return y

    q = turn(s["q_pe"].transpose(0, 1)).transpose(0, 1).contiguous()
    cache = _doubles(s)
    rows = s["rows"].to(torch.float64)
    rows[:, LATENT:] = turn(s["rows"][:, LATENT:])
    if c["kv"] == "e4m3":
        rows = (rows / s["kv_scale"]).clamp(-448.0, 448.0)
    table, t = s["table"].tolist(), 0
    place = []
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        place += [table[b][k // PAGE] * PAGE + k % PAGE for k in range(n - m, n)]
    cache.view(-1, ROW)[torch.tensor(place, device="cuda")] = rows
    return q, cache


def _exact_commit(s):
    cache, table = _doubles(s), s["table"].tolist()
    flat = cache.view(cache.shape[0], -1, ROW)
    paths, counts = s["path"].tolist(), s["count"].tolist()
    lens, frm, to = [], [], []
    for b, (m, n) in enumerate(zip(s["new"], s["total"])):
        place = lambda t: table[b][t // PAGE] * PAGE + t % PAGE  # noqa: E731,B023
        for k in range(counts[b]):
            frm.append(place(n - m + paths[b][k]))
            to.append(place(n - m + k))
        lens.append(n - m + counts[b])
    flat[:, torch.tensor(to, device="cuda")] = flat[:, torch.tensor(frm, device="cuda")]
    return _i32(lens), cache


def _exact_fork(s):
    table, refs = s["table"].tolist(), s["refs"].tolist()
    cache = _doubles(s)
    src, rows, copies = s["src"].tolist(), [], []
    for f in src:
        full = s["total"][f] // PAGE
        for page in table[f][:full]:
            refs[page] += 1
    free = iter([i for i, r in enumerate(refs) if r == 0])
    for f in src:
        full, tail = divmod(s["total"][f], PAGE)
        row = table[f][:full]
        if tail:
            page = next(free)
            refs[page] = 1
            copies.append((table[f][full], page, tail))
            row = row + [page]
        rows.append(row + [-1] * (len(table[f]) - len(row)))
    for old, page, tail in copies:
        cache[:, page, :tail] = cache[:, old, :tail]
    return _i32(rows), _i32(refs), cache


def _exact_resize(s):
    table, refs, lens = s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist()
    rows = []
    for row, n in zip(table, lens):
        need = -(-n // PAGE)
        for page in row[need:]:
            if page >= 0:
                refs[page] -= 1
        rows.append(row[:need] + [-1] * (len(row) - need))
    free = (i for i, r in enumerate(list(refs)) if r == 0)
    for row, n in zip(rows, lens):
        for k in range(-(-n // PAGE)):
            if row[k] < 0:
                row[k] = next(free)
                refs[row[k]] = 1
    return _i32(rows), _i32(refs)
