"""GPU parity of mla_decode_tree and mla_tree_commit against the float64
oracle: trees, forests, chains and stars of any size up to the limit, across
page borders, over contexts cut into pieces, both cache types; rows of accepted
nodes bit for bit."""
import numpy as np
import pytest

import chunk_cases as K
import oracle
import tree_cases as TC

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SENTINEL = 7.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_mla_decode_09_gb300 as mla
    from paged_mla_decode_09_gb300.build import build_library

    build_library()
    mla.load_library()


class Run:
    """Device copies of a case, with outputs and a workspace full of garbage."""

    def __init__(self, c, parents):
        import paged_mla_decode_09_gb300 as mla

        self.c = c
        self.qn, self.qp = K.to_cuda(c.q_nope), K.to_cuda(c.q_pe)
        self.cache, self.table = K.to_cuda(c.kv_cache), K.to_cuda(c.page_table)
        self.lens, self.cu, self.parents = K.to_cuda(c.seq_lens), K.to_cuda(c.cu), K.to_cuda(parents)
        self.out = torch.full(self.qn.shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full(self.qn.shape[:2], SENTINEL, dtype=torch.float32, device="cuda")
        dims = mla.make_prefill_dims(self.qn, self.cache, self.table, self.lens)
        self.ws = torch.full((mla.mla_decode_tree_workspace_size(dims),), 0xFF, dtype=torch.uint8, device="cuda")

    def launch(self, stream=None):
        import paged_mla_decode_09_gb300 as mla

        c = self.c
        mla.mla_decode_tree(self.qn, self.qp, self.cache, self.table, self.lens, self.cu, self.parents, c.scale,
                            c.kv_scale, self.out, self.lse, self.ws, stream)

    def result(self):
        import paged_mla_decode_09_gb300 as mla

        torch.cuda.synchronize()
        status = mla.mla_query_status(self.ws)
        assert not status & (mla.MLA_DEV_TIMEOUT | mla.MLA_DEV_INTERNAL), mla.timeout_diagnostics(self.ws)
        return self.out.float().cpu().numpy().astype(np.float64), self.lse.cpu().numpy().astype(np.float64), status


def check_nodes(c, parents, out, lse, requests=None):
    for b in range(len(c.seq_lens)) if requests is None else requests:
        q0, q1 = int(c.cu[b]), int(c.cu[b + 1])
        for i in range(q1 - q0):
            keys = oracle.tree_keys(int(c.seq_lens[b]), parents[q0:q1], i)
            ref, rl, to, tl = TC.error_bounds(c, b, i, keys)
            eo, el = np.abs(out[q0 + i] - ref), np.abs(lse[q0 + i] - rl)
            assert np.all(eo <= to), (b, i, float((eo / to).max()))
            assert np.all(el <= tl), (b, i, float((el / tl).max()))


def run_and_check(c, parents):
    r = Run(c, parents)
    r.launch()
    out, lse, status = r.result()
    assert status == 0
    n = int(c.cu[-1])
    assert np.all(out[n:] == SENTINEL) and np.all(lse[n:] == SENTINEL)
    check_nodes(c, parents, out, lse)
    return r


CASES = {
    "one_node": dict(new=[1], total=[1], heads=16),
    "one_node_later": dict(new=[1], total=[65], heads=1),
    "page_edges": dict(new=[1, 63, 64, 65], total=[64, 64, 128, 129], heads=4),
    "tree_begins_at_pages": dict(new=[8, 8, 8, 8], total=[71, 72, 73, 136], heads=16),
    "tree_is_all": dict(new=[70, 200], total=[70, 200], heads=4),
    "largest": dict(new=[256], total=[300], heads=3),
    "largest_over_five_pages": dict(new=[256, 255], total=[1000 + 33, 255 + 64], heads=2),
    "odd_heads_no_nodes": dict(new=[0, 5, 0, 30, 0], total=[70, 200, 1, 500, 0], heads=20),
    "wide_heads": dict(new=[3, 17], total=[130, 1000], heads=128),
    "more_heads_than_rows": dict(new=[2], total=[300], heads=200),
    "pieces": dict(new=[9], total=[20000], heads=16),
    "pieces_of_few": dict(new=[6, 4], total=[9000, 2000], heads=64),
    "many_requests": dict(new=[1 + k % 9 for k in range(150)], total=[40 + 7 * k for k in range(150)], heads=8),
    "beyond_the_small_schedule": dict(new=[1 + k % 3 for k in range(600)], total=[4 + k % 70 for k in range(600)], heads=2),
    "full_blocks_pieces": dict(new=[40, 64], total=[6000, 65], heads=32),
    "many_full_blocks": dict(new=[33] * 8 + [7], total=[90 + 83 * k for k in range(9)], heads=64),
    "rows_behind": dict(new=[9, 3], total=[100, 64], heads=16, extra_q=5),
}


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("name", list(CASES))
def test_tree_parity(name, kv_dtype):
    run_and_check(*TC.make(seed=len(name), kv_dtype=kv_dtype, **CASES[name]))


@pytest.mark.parametrize("kind", ["forest", "star", "none"])
@pytest.mark.parametrize("heads", [16, 128])
def test_shapes_of_trees(kind, heads):
    run_and_check(*TC.make([1, 12, 70, 130], [50, 75, 200, 330], heads=heads, kind=kind, seed=heads))


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("heads", [16, 64])
def test_a_chain_is_a_prompt_chunk_bit_for_bit(heads, kv_dtype):
    import paged_mla_decode_09_gb300 as mla

    c, parents = TC.make([5, 100, 0, 256], [900, 100, 7, 700], heads=heads, kind="chain", kv_dtype=kv_dtype, seed=heads)
    r = run_and_check(c, parents)
    out, lse = torch.full_like(r.out, SENTINEL), torch.full_like(r.lse, SENTINEL)
    ws = torch.empty(mla.mla_prefill_workspace_size(mla.make_prefill_dims(r.qn, r.cache, r.table, r.lens)),
                     dtype=torch.uint8, device="cuda")
    mla.mla_prefill(r.qn, r.qp, r.cache, r.table, r.lens, r.cu, 0, 0, c.scale, c.kv_scale, out, lse, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, r.out) and torch.equal(lse, r.lse)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("name", list(K.WIDE_SINGLE))
def test_wide_blocks_of_the_single_form(name, kv_dtype):
    c, parents = TC.make(seed=len(name), kv_dtype=kv_dtype, **K.WIDE_SINGLE[name])
    assert K.takes_single_form(c) and K.may_be_cut(c)
    run_and_check(c, parents)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("new,total,heads", [([8], [9000], 16), ([1, 1], [9000, 5000], 120), ([6, 5, 0], [3000, 700, 5], 20),
                                             ([5, 3], [60, 130], 16)])
def test_a_chain_is_a_prompt_chunk_in_the_single_form(new, total, heads, kv_dtype):
    import paged_mla_decode_09_gb300 as mla

    c, parents = TC.make(new, total, heads=heads, kind="chain", kv_dtype=kv_dtype, seed=heads)
    assert K.takes_single_form(c)
    r = run_and_check(c, parents)
    out, lse = torch.full_like(r.out, SENTINEL), torch.full_like(r.lse, SENTINEL)
    ws = torch.empty(mla.mla_prefill_workspace_size(mla.make_prefill_dims(r.qn, r.cache, r.table, r.lens)),
                     dtype=torch.uint8, device="cuda")
    mla.mla_prefill(r.qn, r.qp, r.cache, r.table, r.lens, r.cu, 0, 0, c.scale, c.kv_scale, out, lse, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, r.out) and torch.equal(lse, r.lse)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_peaked_scores(kv_dtype):
    run_and_check(*TC.make([20, 3], [1500, 900], heads=32, kv_dtype=kv_dtype, seed=5, q_gain=10.0))


def test_bad_trees_raise_flags_and_leave_other_requests_alone():
    import paged_mla_decode_09_gb300 as mla

    c, parents = TC.make([3, 5, 2], [100, 200, 90], heads=16, seed=9)
    for node, value in ((4, 1), (4, 9), (4, -2), (3, 0), (3, 2**31 - 1), (7, -2**31)):  # request 1 has the nodes 3 .. 7
        p = parents.copy()
        p[node] = value
        r = Run(c, p)
        r.launch()
        out, lse, status = r.result()
        assert status == mla.MLA_DEV_BAD_TREE, (node, value)
        as_if = p.copy()
        as_if[node] = -1
        check_nodes(c, as_if, out, lse)
    # parents behind the last request are not read
    p = np.concatenate([parents, np.full(4, 99, np.int32)])
    c2, _ = TC.make([3, 5, 2], [100, 200, 90], heads=16, seed=9, extra_q=4)
    r = Run(c2, p)
    r.launch()
    assert r.result()[2] == 0
    # too many nodes: left out
    c, parents = TC.make([3, 257, 2], [100, 300, 90], heads=2, seed=9)
    r = Run(c, parents)
    r.launch()
    out, lse, status = r.result()
    assert status == mla.MLA_DEV_BAD_TREE
    assert np.all(out[3:260] == SENTINEL) and np.all(lse[3:260] == SENTINEL)
    check_nodes(c, parents, out, lse, requests=[0, 2])


def test_bad_lengths_and_pages():
    import paged_mla_decode_09_gb300 as mla

    c, parents = TC.make([3, 5, 2], [100, 200, 90], heads=16, kind="chain", seed=9)
    r = Run(c, parents)
    r.lens[1] = 2  # three of the five nodes are in front of the cache: they see nothing
    r.launch()
    out, lse, status = r.result()
    assert status == mla.MLA_DEV_BAD_SEQ_LEN
    assert np.all(out[3:6] == 0) and np.all(lse[3:6] == -np.inf) and np.all(np.isfinite(out[6:8]))
    check_nodes(c, parents, out, lse, requests=[0, 2])
    r = Run(c, parents)
    r.lens[2] = 10**6
    r.launch()
    assert r.result()[2] & mla.MLA_DEV_BAD_SEQ_LEN
    r = Run(c, parents)
    r.table[1, 1] = -7
    r.launch()
    out, lse, status = r.result()
    assert status == mla.MLA_DEV_BAD_PAGE_ID
    check_nodes(c, parents, out, lse, requests=[0, 2])
    for cu in ([0, 3, 2, 10], [0, 3, 8, 11], [1, 3, 8, 10], [0, -5, 8, 10], [0, 2**31 - 1, 8, 10]):
        r = Run(c, parents)
        r.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        r.launch()
        assert r.result()[2] & mla.MLA_DEV_BAD_QUERY_RANGE, cu


def test_repeats_and_table_slices_are_bit_identical():
    c, parents = TC.make([7, 60, 1], [300, 2000, 5000], heads=32, seed=11)
    r = run_and_check(c, parents)
    out, lse = r.out.clone(), r.lse.clone()
    wide = torch.full((3, c.page_table.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :c.page_table.shape[1]] = r.table
    r.table = wide[:, :c.page_table.shape[1]]
    for _ in range(3):
        r.out.fill_(0)
        r.ws.fill_(0x55)
        r.launch()
        r.result()
        assert torch.equal(r.out, out) and torch.equal(r.lse, lse)


def test_captured_call_follows_its_inputs():
    """A captured call reads lengths, offsets, parents and tables anew; two
    graphs that share a workspace run one after the other."""
    a, pa = TC.make([6, 2, 9], [500, 64, 1300], heads=16, seed=21)
    b, pb = TC.make([1, 15, 1], [33, 1000, 700], heads=16, seed=22)
    width = max(a.page_table.shape[1], b.page_table.shape[1])
    r = Run(a, pa)
    r.table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    r.cache = torch.zeros((max(a.kv_cache.shape[0], b.kv_cache.shape[0]), 64, 576), dtype=torch.bfloat16, device="cuda")
    graphs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            r.launch()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.launch()
        graphs.append(g)
    for k, (c, p) in enumerate(((a, pa), (b, pb), (a, pa))):
        r.table.fill_(-1)
        r.table[:, :c.page_table.shape[1]] = K.to_cuda(c.page_table)
        r.cache[:c.kv_cache.shape[0]] = K.to_cuda(c.kv_cache)
        r.lens.copy_(K.to_cuda(c.seq_lens))
        r.cu.copy_(K.to_cuda(c.cu))
        for dst, src in ((r.qn, c.q_nope), (r.qp, c.q_pe), (r.parents, p)):
            src = K.to_cuda(src)
            n = min(dst.shape[0], src.shape[0])
            dst.zero_()
            dst[:n] = src[:n]
        graphs[k % 2].replay()
        graphs[(k + 1) % 2].replay()
        out, lse, status = r.result()
        assert status == 0
        check_nodes(c, p, out, lse)


def test_streams_with_their_own_workspaces():
    rs = [run_and_check(*TC.make([50], [1500], heads=16, seed=31)), run_and_check(*TC.make([3, 3], [4000, 200], heads=64, seed=32))]
    want = [(r.out.clone(), r.lse.clone()) for r in rs]
    streams = [torch.cuda.Stream() for _ in rs]
    torch.cuda.synchronize()
    for _ in range(5):
        for r, s in zip(rs, streams):
            r.launch(s)
    torch.cuda.synchronize()
    for r, (o, l) in zip(rs, want):
        assert torch.equal(r.out, o) and torch.equal(r.lse, l)


# ------------------------------------------------------------------- commit
def commit_case(rng, nodes, totals, layers, dtype, cols=None):
    """Random rows, ascending paths, a pool with the pages in random order."""
    B = len(nodes)
    width = max(-(-t // 64) for t in totals) + 1
    count = sum(-(-t // 64) for t in totals) + 2
    ids = rng.permutation(count).astype(np.int32)
    table, at = np.full((B, width), -1, np.int32), 0
    for b, t in enumerate(totals):
        n = -(-t // 64)
        table[b, :n] = ids[at:at + n]
        at += n
    top = 1 << (8 if dtype == np.uint8 else 16)
    cache = rng.integers(0, top, size=(layers, count, 64, 576)).astype(dtype)
    cols = cols or max(max(nodes), 1)
    path, num = np.full((B, cols), -1, np.int32), np.zeros(B, np.int32)
    for b, n in enumerate(nodes):
        k = int(rng.integers(0, min(n, cols) + 1))
        path[b, :k] = np.sort(rng.permutation(n)[:k])
        num[b] = k
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    return cache, table, np.asarray(totals, np.int32), cu, path, num


def gpu_commit(cache, table, lens, cu, path, num):
    import paged_mla_decode_09_gb300 as mla

    dev = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (table, lens, cu, path, num)]
    t = torch.from_numpy(cache.view(np.int16) if cache.dtype == np.uint16 else cache).cuda()
    t = t.view(torch.bfloat16) if cache.dtype == np.uint16 else t
    new_lens = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_tree_commit(t, *dev, new_lens, status)
    torch.cuda.synchronize()
    raw = t.view(torch.int16).cpu().numpy().view(np.uint16) if cache.dtype == np.uint16 else t.cpu().numpy()
    return raw, new_lens.cpu().numpy(), int(status.item())


@pytest.mark.parametrize("dtype", [np.uint16, np.uint8])
@pytest.mark.parametrize("nodes,extra,layers", [([1], 0, 1), ([8], 60, 3), ([0, 5, 256, 70], 0, 1),
                                                ([33] * 20, 100, 9), ([3, 64, 1, 17, 0], 127, 5)])
def test_commit_moves_rows(nodes, extra, layers, dtype):
    rng = np.random.default_rng(len(nodes) + layers)
    for _ in range(4):
        case = commit_case(rng, nodes, [n + int(rng.integers(0, extra + 1)) for n in nodes], layers, dtype)
        raw, lens, status = gpu_commit(*case)
        ref, ref_lens = oracle.tree_commit_ref(*case)
        assert status == 0
        assert np.array_equal(lens, ref_lens) and np.array_equal(raw, ref)


def test_commit_leaves_out_what_is_wrong():
    import paged_mla_decode_09_gb300 as mla

    rng = np.random.default_rng(5)
    case = commit_case(rng, [6, 9, 7], [70, 140, 64], 2, np.uint16)
    case[4][:] = -1
    for b in range(3):
        case[4][b, :3] = [0, 2, 5]
    case[5][:] = 3
    ref, ref_lens = oracle.tree_commit_ref(*case)

    def broken(what, flag):
        bad = [np.array(a, copy=True) for a in case]
        what(bad)
        raw, lens, status = gpu_commit(*bad)
        assert status == flag
        good = [np.array(a, copy=True) for a in case]
        good[5][1] = 0  # request 1 left out
        want, _ = oracle.tree_commit_ref(*good)
        assert np.array_equal(raw, want)
        assert lens[[0, 2]].tolist() == ref_lens[[0, 2]].tolist() and lens[1] == bad[2][1]

    def put(i, at, v):
        return lambda a: a[i].__setitem__(at, v)

    for row in ([0, 5, 2], [0, 0, 1], [0, 2, 9], [-1, 2, 5], [2, 1, 5], [0, 2, 2**31 - 1]):
        broken(lambda a, row=row: a[4].__setitem__((1, slice(0, 3)), row), mla.MLA_DEV_BAD_INDEX)
    broken(put(5, 1, 10), mla.MLA_DEV_BAD_INDEX)
    broken(put(5, 1, -1), mla.MLA_DEV_BAD_INDEX)
    broken(put(2, 1, 8), mla.MLA_DEV_BAD_SEQ_LEN)
    broken(put(2, 1, 10**6), mla.MLA_DEV_BAD_SEQ_LEN)
    # a bad page id: that move alone is skipped (node 5 of request 0 is in slot 69, its second page)
    bad = [np.array(a, copy=True) for a in case]
    bad[1][0, 1] = 99
    raw, lens, status = gpu_commit(*bad)
    assert status == mla.MLA_DEV_BAD_PAGE_ID and np.array_equal(lens, ref_lens)
    assert np.array_equal(raw[:, case[1][1]], ref[:, case[1][1]])


def test_commit_over_strided_layers_and_captured():
    import paged_mla_decode_09_gb300 as mla

    rng = np.random.default_rng(8)
    cache, table, lens, cu, path, num = commit_case(rng, [16] * 4, [80, 90, 100, 16], 6, np.uint8)
    wide = torch.zeros((6, cache.shape[1] + 3, 64, 576), dtype=torch.uint8, device="cuda")
    t = wide[:, :cache.shape[1]]
    t.copy_(torch.from_numpy(cache))
    dev = [torch.from_numpy(a).cuda() for a in (table, lens, cu, path, num)]
    new_lens, status = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_tree_commit(t, *dev, new_lens, status)
    g.replay()
    torch.cuda.synchronize()
    ref, ref_lens = oracle.tree_commit_ref(cache, table, lens, cu, path, num)
    assert np.array_equal(t.cpu().numpy(), ref) and np.array_equal(new_lens.cpu().numpy(), ref_lens)
    dev[4].zero_()  # a replay reads the counts anew: nothing accepted
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(t.cpu().numpy(), ref) and np.array_equal(new_lens.cpu().numpy(), lens - 16)
    assert status.item() == 0
