"""Entry points as the first CUDA call of a thread, where the runtime has no
context current yet: they give what they give in the main thread.  And as the
process's first call, captured."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_mla_decode_09_gb300 as mla
    from paged_mla_decode_09_gb300.build import build_library

    build_library()
    mla.load_library()


def calls():
    """name -> (call, outputs); two requests of 700 and 650 tokens."""
    import paged_mla_decode_09_gb300 as mla

    g = torch.Generator("cuda").manual_seed(3)

    def bf(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def i32(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def ws(n):
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    B, H = 2, 64
    cache, table = bf(22, 64, 576), torch.randperm(22, generator=g, device="cuda").to(torch.int32).view(B, 11)
    seq = cache, table, i32([700, 650])
    qn, qp, out, lse = bf(B, 1, H, 512), bf(B, 1, H, 64), bf(B, 1, H, 512), torch.zeros(B, 1, H, device="cuda")
    tn, tp, tout, tlse = bf(6, H, 512), bf(6, H, 64), bf(6, H, 512), torch.zeros(6, H, device="cuda")
    d, dt = mla.make_dims(qn, cache, table), mla.make_prefill_dims(tn, *seq)
    cu, parents = i32([0, 2, 6]), i32([-1, 0, -1, 0, 0, 1])
    shared = table.clone()
    shared[1, :3] = shared[0, :3]
    picks = torch.randperm(600, generator=g, device="cuda")[:80].to(torch.int32).view(B, 1, 40)
    offsets, gathered = torch.tensor([0, 700], device="cuda"), bf(1350, 576)
    mass, fixed, status = torch.zeros(B, 704, device="cuda"), torch.full((B, 1, H), 6.0, device="cuda"), i32([0])
    rows, plan, written = bf(6, 576), mla.mla_rope_plan(64), cache.clone()
    refs, t2, r2 = torch.ones(22, dtype=torch.int32, device="cuda"), torch.zeros_like(table), i32([0] * 22)
    large, counts = torch.full((40, 600), -1, dtype=torch.int32, device="cuda"), torch.zeros(30000, dtype=torch.int32, device="cuda")
    lt, lc, lens = torch.zeros_like(large), torch.zeros_like(counts), i32([300 * k for k in range(40)])
    w1, w2, w3 = (ws(mla.mla_decode_workspace_size(d)), ws(mla.mla_decode_window_workspace_size(d)),
                  ws(mla.mla_decode_sparse_workspace_size(d, 40)))
    w4, w5, w6 = (ws(mla.mla_decode_cascade_workspace_size(d, 3)), ws(mla.mla_prefill_workspace_size(dt)),
                  ws(mla.mla_decode_tree_workspace_size(dt)))
    w7, w8, w9 = (ws(mla.mla_attn_mass_workspace_size(d)), ws(mla.mla_page_resize_workspace_size(40, 600, 30000)),
                  ws(mla.mla_page_fork_workspace_size(B, B, 11, 22)))
    src, full, lib = i32([1, 0]), i32([704, 640]), mla.load_library()
    q_out = tout.view(-1)[:6 * H * 64].view(6, H, 64)

    def noalloc():
        p = [ctypes.c_void_p(t.data_ptr()) for t in (qn, qp, *seq, out, lse, status)]
        assert lib.mla_decode_noalloc(ctypes.byref(d), *p[:5], 1, 0.07, 1.0, *p[5:], None) == 0

    return {
        "decode": (lambda: mla.mla_decode(qn, qp, *seq, 1, 0.07, 1.0, out, lse, w1), [out, lse]),
        "noalloc": (noalloc, [out, lse]),
        "gather": (lambda: mla.mla_gather_rows(*seq, offsets, gathered, w1), [gathered]),
        "window": (lambda: mla.mla_decode_window(qn, qp, *seq, 200, 3, 0.07, 1.0, out, lse, w2), [out, lse]),
        "sparse": (lambda: mla.mla_decode_sparse(qn, qp, *seq, picks, 0.07, 1.0, out, lse, w3), [out, lse]),
        "cascade": (lambda: mla.mla_decode_cascade(qn, qp, cache, shared, seq[2], 3, 0.07, 1.0, out, lse, w4), [out, lse]),
        "prefill": (lambda: mla.mla_prefill(tn, tp, *seq, cu, 0, 0, 0.07, 1.0, tout, tlse, w5), [tout, tlse]),
        "tree": (lambda: mla.mla_decode_tree(tn, tp, *seq, cu, parents, 0.07, 1.0, tout, tlse, w6), [tout, tlse]),
        "mass": (lambda: mla.mla_attn_mass(qn, qp, *seq, fixed, 0, 0.07, 1.0, None, mass, w7), [mass]),
        "rope": (lambda: mla.mla_rope_pack(plan, tp, rows, None, table, seq[2], cu, 1.0, q_out, written, status),
                 [q_out]),
        "resize": (lambda: mla.mla_page_resize(lens, large, counts, lt, lc, w8), [lt, lc]),
        "fork": (lambda: mla.mla_page_fork(src, full, table, refs, written, t2, r2, w9), [t2, r2]),
    }


@pytest.mark.parametrize("name", ["decode", "noalloc", "gather", "window", "sparse", "cascade", "prefill", "tree", "mass",
                                  "rope", "resize", "fork"])
def test_a_threads_first_call(name):
    call, outs = calls()[name]
    call()  # launch shapes and kernels are known from here on: the thread's call asks the driver for little
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    failed = []

    def run():
        try:
            call()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and any(bool(w.any()) for w in want)


def test_threads_at_once():
    """Decodes, trees and page calls from threads of their own, on streams of their own."""
    jobs = [calls()[n] for n in ("decode", "tree", "prefill", "mass", "resize")]
    want = []
    for call, outs in jobs:
        call()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    streams, failed = [torch.cuda.Stream() for _ in jobs], []

    def run(call, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(50):
                    call()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(c, s)) for (c, _), s in zip(jobs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for (_, outs), ref in zip(jobs, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_first_calls_of_a_process_can_be_captured():
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "first_capture_speculative_child.py")
    r = subprocess.run([sys.executable, child], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
