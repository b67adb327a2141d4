"""Child process of test_gpu_new_calls_extremes: each operator's first call of
the process is captured into a CUDA graph, replayed, and compared with an
eager call.  Exit code 0 when all agree.

Usage: python tests/first_capture_child.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import paged_mla_decode_09_gb300 as mla  # noqa: E402

mla.load_library()
gen = torch.Generator(device="cuda")
gen.manual_seed(1)
B, H, L, pages = 2, 64, 700, 22
cache = torch.randn(pages, 64, 576, generator=gen, device="cuda").bfloat16()
table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(B, 11)
lens = torch.tensor([L, L - 9], dtype=torch.int32, device="cuda")
ok = True


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


for Q in (1, 3):
    qn = torch.randn(B, Q, H, 512, generator=gen, device="cuda").bfloat16()
    qp = torch.randn(B, Q, H, 64, generator=gen, device="cuda").bfloat16()
    out, lse = torch.zeros_like(qn), torch.zeros(B, Q, H, device="cuda")
    mass = torch.zeros(B, 704, device="cuda")
    mws = torch.zeros(mla.mla_attn_mass_workspace_size(mla.make_dims(qn, cache, table)), dtype=torch.uint8, device="cuda")
    wws = torch.zeros(mla.mla_decode_window_workspace_size(mla.make_dims(qn, cache, table)), dtype=torch.uint8,
                      device="cuda")
    fixed = torch.full((B, Q, H), 6.0, device="cuda")
    captured(f"mass, {Q} tokens", lambda: mla.mla_attn_mass(qn, qp, cache, table, lens, fixed, 0, 0.07, 1.0, None, mass,
                                                            mws), [mass])
    captured(f"window, {Q} tokens", lambda: mla.mla_decode_window(qn, qp, cache, table, lens, 200, 3, 0.07, 1.0, out,
                                                                  lse, wws), [out, lse])
cu = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
q3, p3, o3, l3 = qn.view(6, H, 512), qp.view(6, H, 64), out.view(6, H, 512), lse.view(6, H)
pws = torch.zeros(mla.mla_prefill_workspace_size(mla.make_prefill_dims(q3, cache, table, lens)), dtype=torch.uint8,
                  device="cuda")
captured("prefill", lambda: mla.mla_prefill(q3, p3, cache, table, lens, cu, 0, 0, 0.07, 1.0, o3, l3, pws), [o3, l3])
new, kept, mo = lens.clone(), torch.zeros(B, 300, dtype=torch.int32, device="cuda"), torch.zeros_like(mass)
ews = torch.zeros(mla.mla_evict_workspace_size(B, 300), dtype=torch.uint8, device="cuda")
start = cache.clone()


def evict():
    cache.copy_(start)
    mla.mla_evict(mass, None, lens, table, cache, 300, 4, 50, new, kept, mo, None, ews)


captured("evict", evict, [new, kept, mo])
sys.exit(0 if ok else 1)
