"""The calls of a speculative step at the ends of what their headers allow:
offsets that pass 32 bits, the largest and smallest sizes, many requests, calls
at once, and buffers behind what a call may write."""
import numpy as np
import pytest

import oracle
import tree_cases as TC

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BIG_POOL = 66000  # pages: 2.4e9 values, 4.9e9 bytes of bf16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_mla_decode_09_gb300 as mla
    from paged_mla_decode_09_gb300.build import build_library

    build_library()
    mla.load_library()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def bf(*shape, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


@pytest.fixture(scope="module")
def pool():
    return torch.zeros((BIG_POOL, 64, 576), dtype=torch.bfloat16, device="cuda")


def test_rows_move_behind_32_bits(pool):
    """Pages at both ends of a pool of 4.9 GB: written, attended to, moved, copied."""
    import paged_mla_decode_09_gb300 as mla

    first = BIG_POOL - 3
    table = i32([[BIG_POOL - 1, first], [0, 1]])
    lens, cu = i32([70, 70]), i32([0, 70, 140])
    rows, q = bf(140, 576, seed=1), bf(140, 2, 64, seed=2)
    status = i32([0])
    q_out = torch.empty_like(q)
    mla.mla_rope_pack(mla.mla_rope_plan(64), q, rows, None, table, lens, cu, 1.0, q_out, pool, status)
    assert torch.equal(pool[BIG_POOL - 1, :, :512], rows[:64, :512]) and torch.equal(pool[first, :6, :512], rows[64:70, :512])
    assert torch.equal(pool[0, :, :512], rows[70:134, :512])
    # a tree over the same pages, where requests with equal rows see equal things
    pool[0].copy_(pool[BIG_POOL - 1])
    pool[1].copy_(pool[first])
    parents, qn = i32([-1, 0, 0, 1] * 2), bf(4, 2, 512, seed=3).repeat(2, 1, 1)
    qp, cu4 = bf(4, 2, 64, seed=4).repeat(2, 1, 1), i32([0, 4, 8])
    out, lse = torch.zeros_like(qn), torch.zeros((8, 2), device="cuda")
    ws = torch.empty(mla.mla_decode_tree_workspace_size(mla.make_prefill_dims(qn, pool, table, lens)), dtype=torch.uint8,
                     device="cuda")
    mla.mla_decode_tree(qn, qp, pool, table, lens, cu4, parents, 0.1, 1.0, out, lse, ws)
    assert mla.mla_query_status(ws) == 0
    assert torch.equal(out[:4], out[4:]) and torch.equal(lse[:4], lse[4:]) and torch.all(lse > 0)
    # nodes 0, 2 and 3 stay
    before = pool[first].clone()
    new_lens, num = i32([0, 0]), i32([3, 0])
    mla.mla_tree_commit(pool, table, lens, cu4, i32([[0, 2, 3], [-1, -1, -1]]), num, new_lens, status)
    assert new_lens.tolist() == [69, 66] and torch.equal(pool[first, 3:5], before[4:6])
    # forks between the ends
    refs = torch.zeros(BIG_POOL, dtype=torch.int32, device="cuda")
    refs[table.flatten().long()] = 1
    refs[2:BIG_POOL - 2] = 7
    t2 = torch.full((2, 2), -5, dtype=torch.int32, device="cuda")
    fws = torch.empty(mla.mla_page_fork_workspace_size(2, 2, 2, BIG_POOL), dtype=torch.uint8, device="cuda")
    mla.mla_page_fork(i32([1, -1]), lens, table, refs, pool, t2, refs, fws)
    assert mla.mla_query_status(fws) == 0
    assert t2.tolist() == [[0, BIG_POOL - 2], [-1, -1]] and refs[0] == 2 and refs[BIG_POOL - 2] == 1
    assert torch.equal(pool[BIG_POOL - 2, :6], pool[1, :6])
    assert status.item() == 0


def test_layers_lie_more_than_32_bits_apart(pool):
    import paged_mla_decode_09_gb300 as mla

    layers = pool.view(2, BIG_POOL // 2, 64, 576)
    layers[:, 7] = bf(2, 64, 576, seed=5)
    want = layers[:, 7, 40].clone()
    status, new_lens = i32([0]), i32([0])
    mla.mla_tree_commit(layers, i32([[7]]), i32([41]), i32([0, 9]), i32([[8]]), i32([1]), new_lens, status)
    assert new_lens.tolist() == [33] and status.item() == 0 and torch.equal(layers[:, 7, 32], want)
    refs = torch.ones(BIG_POOL // 2, dtype=torch.int32, device="cuda")
    refs[BIG_POOL // 2 - 1] = 0
    out = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    ws = torch.empty(mla.mla_page_fork_workspace_size(1, 1, 1, BIG_POOL // 2), dtype=torch.uint8, device="cuda")
    mla.mla_page_fork(i32([0]), i32([33]), i32([[7]]), refs, layers, out, refs, ws)
    assert out.tolist() == [[BIG_POOL // 2 - 1]] and torch.equal(layers[:, -1, :33], layers[:, 7, :33])


def test_probabilities_behind_32_bits():
    import paged_mla_decode_09_gb300 as mla

    step, v = (1 << 31) + 64, 3000  # elements between rows
    big = torch.zeros(2 * step + v, device="cuda")
    target = big.as_strided((3, v), (step, 1))
    rng = np.random.default_rng(1)
    p = rng.dirichlet(np.ones(v), 3).astype(np.float32)
    target.copy_(torch.from_numpy(p))
    tokens = i32([0, int(p[0].argmax()), int(p[1].argmax())])
    parents, cu = i32([-1, 0, 1]), i32([0, 3])
    accept, sample = torch.zeros(3, device="cuda"), torch.full((1,), 0.7, device="cuda")
    path, out, num, status = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 3), (1, 3), (1,), (1,)))
    mla.mla_verify(target, target, tokens, parents, cu, accept, sample, path, out, num, status)
    want = oracle.verify_ref(p, p, tokens.tolist(), parents.tolist(), [0, 3], [0.0] * 3, [float(np.float32(0.7))], 3)
    assert np.array_equal(path.cpu().numpy(), want[0]) and np.array_equal(out.cpu().numpy(), want[1])
    assert num.tolist() == [3] and status.item() == 0


def test_many_requests():
    """More requests than blocks run at once, of one node each."""
    import paged_mla_decode_09_gb300 as mla

    B, v = 3000, 37
    rng = np.random.default_rng(2)
    p = rng.dirichlet(np.ones(v), B).astype(np.float32)
    cu = np.arange(B + 1, dtype=np.int32)
    accept, sample = rng.random(B).astype(np.float32), rng.random(B).astype(np.float32)
    path, out, num = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, 2), (B, 2), (B,)))
    status = i32([0])
    mla.mla_verify(torch.from_numpy(p).cuda(), None, i32([0] * B), i32([-1] * B), torch.from_numpy(cu).cuda(),
                   torch.from_numpy(accept).cuda(), torch.from_numpy(sample).cuda(), path, out, num, status)
    want = oracle.verify_ref(p, None, [0] * B, [-1] * B, cu, accept, sample, 2)
    assert np.array_equal(out.cpu().numpy(), want[1]) and np.array_equal(num.cpu().numpy(), want[2]) and status.item() == 0
    # rows of two columns, each a page more or less
    cols, pages = 2, 7000
    lens = rng.integers(0, 129, B)
    table, refs = np.full((B, cols), -1, np.int32), np.zeros(pages, np.int32)
    ws = torch.empty(mla.mla_page_resize_workspace_size(B, cols, pages), dtype=torch.uint8, device="cuda")
    t, r = i32(table), i32(refs)
    for k in range(3):
        want_t, want_r, st = oracle.page_resize_ref(lens, table, refs)
        mla.mla_page_resize(i32(lens), t, r, t, r, ws)
        assert st == 0 and mla.mla_query_status(ws) == 0
        assert np.array_equal(t.cpu().numpy(), want_t) and np.array_equal(r.cpu().numpy(), want_r)
        table, refs = want_t, want_r
        lens = rng.integers(0, 129, B)
    # as many rows moved, in two layers
    cache = torch.randint(0, 256, (2, pages, 64, 576), dtype=torch.uint8, device="cuda")
    cu2 = np.cumsum(np.concatenate([[0], np.minimum(lens, 2)])).astype(np.int32)
    want_t, want_r, _ = oracle.page_resize_ref(lens, table, refs)
    n = np.diff(cu2)
    path = np.where(n == 2, 1, 0).astype(np.int32)[:, None]
    num = (n > 0).astype(np.int32)
    ref, ref_lens = oracle.tree_commit_ref(cache.cpu().numpy(), want_t, lens, cu2, path, num)
    new_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    mla.mla_tree_commit(cache, i32(want_t), i32(lens), i32(cu2), i32(path), i32(num), new_lens, status)
    assert np.array_equal(new_lens.cpu().numpy(), ref_lens) and np.array_equal(cache.cpu().numpy(), ref)
    assert status.item() == 0


def test_guards_around_the_outputs_stay():
    """Outputs that end where another buffer begins."""
    import paged_mla_decode_09_gb300 as mla

    def guarded(n, t=torch.int32):
        whole = torch.full((n + 64,), 77, dtype=t, device="cuda")
        return whole, whole[32:32 + n]

    rng = np.random.default_rng(4)
    B, T, v, cols = 5, 20, 1001, 3
    parents = sum([TC.random_tree(rng, 4) for _ in range(B)], [])
    p = torch.softmax(torch.randn(T, v, device="cuda"), dim=1)
    bufs = [guarded(B * cols), guarded(B * cols), guarded(B), guarded(1)]
    bufs[3][1].zero_()
    mla.mla_verify(p, p, i32(rng.integers(0, v, T)), i32(parents), i32(range(0, T + 1, 4)), torch.rand(T, device="cuda"),
                   torch.rand(B, device="cuda"), bufs[0][1].view(B, cols), bufs[1][1].view(B, cols), bufs[2][1], bufs[3][1])
    for whole, mine in bufs:
        assert torch.all(whole[:32] == 77) and torch.all(whole[32 + mine.numel():] == 77)
    t, r = guarded(B * 7), guarded(33)
    ws = torch.full((mla.mla_page_resize_workspace_size(B, 7, 33) + 4096,), 77, dtype=torch.uint8, device="cuda")
    n = mla.mla_page_resize_workspace_size(B, 7, 33)
    mla.mla_page_resize(i32([0, 64, 65, 448, 300]), torch.full((B, 7), -1, dtype=torch.int32, device="cuda"),
                        torch.zeros(33, dtype=torch.int32, device="cuda"), t[1].view(B, 7), r[1], ws[:n])
    for whole, mine in (t, r):
        assert torch.all(whole[:32] == 77) and torch.all(whole[32 + mine.numel():] == 77)
    assert torch.all(ws[n:] == 77)
    # the tree's workspace
    c, par = TC.make([9, 30, 1], [200, 30, 4000], heads=16, seed=3)
    import chunk_cases as K

    qn, qp, cache, table = (K.to_cuda(a) for a in (c.q_nope, c.q_pe, c.kv_cache, c.page_table))
    lens, cu = K.to_cuda(c.seq_lens), K.to_cuda(c.cu)
    n = mla.mla_decode_tree_workspace_size(mla.make_prefill_dims(qn, cache, table, lens))
    ws = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(qn), torch.zeros(qn.shape[:2], device="cuda")
    mla.mla_decode_tree(qn, qp, cache, table, lens, cu, K.to_cuda(par), c.scale, 1.0, out, lse, ws[:n])
    assert mla.mla_query_status(ws) == 0 and torch.all(ws[n:] == 77)
    with pytest.raises(mla.MlaError):
        mla.mla_decode_tree(qn, qp, cache, table, lens, cu, K.to_cuda(par), c.scale, 1.0, out, lse, ws[:n - 256])


def test_calls_at_once():
    """The page calls of two pools, verifications and a rotation on four
    streams, again and again; each gives what it gives alone."""
    import paged_mla_decode_09_gb300 as mla

    rng = np.random.default_rng(5)
    jobs = []
    for k in range(2):
        B, cols, pages = 40, 600, 30000
        lens = i32(rng.integers(0, cols * 64, B) // 2)
        t, r = torch.full((B, cols), -1, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
        to, ro = torch.empty_like(t), torch.empty_like(r)
        ws = torch.empty(mla.mla_page_resize_workspace_size(B, cols, pages), dtype=torch.uint8, device="cuda")
        jobs.append((lambda s, a=(lens, t, r, to, ro, ws): mla.mla_page_resize(*a, stream=s), (to, ro)))
    p = torch.softmax(4 * torch.randn(48, 20011, device="cuda"), dim=1)
    path, out = torch.zeros((8, 6), dtype=torch.int32, device="cuda"), torch.zeros((8, 6), dtype=torch.int32, device="cuda")
    num, st = torch.zeros(8, dtype=torch.int32, device="cuda"), i32([0])
    args = (p, p, i32(rng.integers(0, 20011, 48)), i32([-1, 0, 1, 2, 3, 4] * 8), i32(range(0, 49, 6)),
            torch.rand(48, device="cuda"), torch.rand(8, device="cuda"), path, out, num, st)
    jobs.append((lambda s: mla.mla_verify(*args, stream=s), (path, out, num)))
    q, rows = bf(900, 32, 64, seed=7), bf(900, 576, seed=8)
    q_out, cache = torch.empty_like(q), torch.zeros((20, 64, 576), dtype=torch.uint8, device="cuda")
    plan, st2 = mla.mla_rope_plan(64, interleaved=False), i32([0])
    rope = (plan, q, rows, None, i32([range(20)]), i32([1000]), i32([0, 900]), 0.02, q_out, cache, st2)
    jobs.append((lambda s: mla.mla_rope_pack(*rope, stream=s), (q_out, cache)))
    torch.cuda.synchronize()
    want = []
    for call, outs in jobs:
        call(None)
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        for o in outs:
            o.zero_()
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (call, _), s in zip(jobs, streams):
            call(s)
    torch.cuda.synchronize()
    for (_, outs), ref in zip(jobs, want):
        assert all(torch.equal(o, r) for o, r in zip(outs, ref))
    assert st.item() == 0 and st2.item() == 0
