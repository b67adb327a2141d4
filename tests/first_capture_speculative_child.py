"""Child process of test_gpu_threads: the process's first call of each operator
of a speculative step is captured into a CUDA graph, replayed, and compared
with an eager call.  Exit code 0 when all agree.

Usage: python tests/first_capture_speculative_child.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import paged_mla_decode_09_gb300 as mla  # noqa: E402

mla.load_library()
gen = torch.Generator(device="cuda")
gen.manual_seed(1)
ok = True


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def bf(*shape):
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


def captured(name, fn, outs):
    global ok
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    fn()
    torch.cuda.synchronize()
    same = all(torch.equal(a, b) for a, b in zip(got, outs)) and all(bool(a.float().abs().sum() > 0) for a in got)
    print(name, same)
    ok = ok and same


H = 16
cache, table, lens, cu = bf(22, 64, 576), torch.arange(22, dtype=torch.int32, device="cuda").view(2, 11), i32([700, 650]), i32([0, 3, 8])
parents, status = i32([-1, 0, 0, -1, 0, 0, 1, 3]), i32([0])
# page calls: the first needs a cluster of 16 blocks, beyond the portable size
big, counts = torch.full((40, 600), -1, dtype=torch.int32, device="cuda"), torch.zeros(30000, dtype=torch.int32, device="cuda")
to, ro = torch.zeros_like(big), torch.zeros_like(counts)
ws = torch.zeros(mla.mla_page_resize_workspace_size(40, 600, 30000), dtype=torch.uint8, device="cuda")
n40, src = i32([37 * k for k in range(40)]), i32([1, 0])
captured("resize, large", lambda: mla.mla_page_resize(n40, big, counts, to, ro, ws), [to, ro])
for pages in (20000, 40):
    pool = torch.zeros((pages, 64, 576), dtype=torch.uint8, device="cuda")
    refs, t2 = torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.zeros_like(table)
    refs[:22] = 1
    r2 = torch.zeros_like(refs)
    fws = torch.zeros(mla.mla_page_fork_workspace_size(2, 2, 11, pages), dtype=torch.uint8, device="cuda")
    captured(f"fork, {pages} pages", lambda: mla.mla_page_fork(src, lens, table, refs, pool, t2, r2, fws), [t2, r2])
small, c2 = torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
t3, r3 = torch.zeros_like(small), torch.zeros_like(c2)
n3 = i32([65, 1])
captured("resize, small", lambda: mla.mla_page_resize(n3, small, c2, t3, r3, ws), [t3, r3])

for heads in (H, 128):  # blocks of 128 and of 256 rows
    qn, qp, out, lse = bf(8, heads, 512), bf(8, heads, 64), bf(8, heads, 512), torch.zeros(8, heads, device="cuda")
    tws = torch.zeros(mla.mla_decode_tree_workspace_size(mla.make_prefill_dims(qn, cache, table, lens)), dtype=torch.uint8,
                      device="cuda")
    captured(f"tree, {heads} heads", lambda: mla.mla_decode_tree(qn, qp, cache, table, lens, cu, parents, 0.07, 1.0, out, lse,
                                                                tws), [out, lse])
rows, q, q_out, written = bf(8, 576), bf(8, H, 64), bf(8, H, 64), torch.zeros_like(cache)
for inter in (True, False):
    plan = mla.mla_rope_plan(64, interleaved=inter)
    captured(f"rope, interleaved {inter}", lambda: mla.mla_rope_pack(plan, q, rows, None, table, lens, cu, 1.0, q_out, written,
                                                                     status), [q_out, written])
p = torch.softmax(4 * torch.randn(8, 5000, generator=gen, device="cuda"), dim=1)
tokens, u = i32([0, 7, 9, 0, 3, 4, 5, 6]), torch.rand(8, generator=gen, device="cuda")
path, toks, num = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 4), (2, 4), (2,)))
for draft in (None, p.roll(1, 1).contiguous()):
    captured(f"verify, draft {draft is not None}", lambda: mla.mla_verify(p, draft, tokens, parents, cu, u, u[:2], path, toks,
                                                                          num, status), [path, toks, num])
new_lens, kept, count = i32([0, 0]), i32([[0, 2], [0, 1]]), i32([2, 2])
captured("commit", lambda: mla.mla_tree_commit(cache, table, lens, cu, kept, count, new_lens, status), [new_lens])
ok = ok and status.item() == 0
sys.exit(0 if ok else 1)
