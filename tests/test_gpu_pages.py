"""mla_page_resize and mla_page_fork against the oracle: tables, counts and
cache rows are whole numbers and bytes, and have to be equal."""
import numpy as np
import pytest

import oracle

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


def pool(rng, lens, cols, pages, share=0.3):
    """Tables of requests of the given lengths, some sharing the beginning of
    the one before, with their counts."""
    ids = rng.permutation(pages).astype(np.int32)
    table, at = np.full((len(lens), cols), -1, np.int32), 0
    for b, n in enumerate(lens):
        k = -(-int(n) // 64)
        table[b, :k] = ids[at:at + k]
        at += k
        if b and rng.random() < share:
            m = min(k, -(-int(lens[b - 1]) // 64)) // 2
            table[b, :m] = table[b - 1, :m]
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    return table, refs


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def resize(lens, table, refs, in_place=False):
    import paged_mla_decode_09_gb300 as mla

    t, r, n = cuda(table), cuda(refs), cuda(np.asarray(lens, np.int32))
    to, ro = (t, r) if in_place else (torch.full_like(t, -5), torch.full_like(r, -5))
    ws = torch.full((mla.mla_page_resize_workspace_size(*table.shape, len(refs)),), 0xFF, dtype=torch.uint8, device="cuda")
    mla.mla_page_resize(n, t, r, to, ro, ws)
    torch.cuda.synchronize()
    return to.cpu().numpy(), ro.cpu().numpy(), mla.mla_query_status(ws)


def check_resize(lens, table, refs):
    want = oracle.page_resize_ref(lens, table, refs)
    for in_place in (False, True):
        got = resize(lens, table, refs, in_place)
        assert got[2] == want[2]
        assert np.array_equal(got[0], want[0]), np.argwhere(got[0] != want[0])[:5].tolist()
        assert np.array_equal(got[1], want[1])
    return want


@pytest.mark.parametrize("B,cols,pages", [(1, 1, 1), (1, 1, 2), (1, 7, 9), (3, 5, 40), (5, 33, 1000), (64, 16, 1024),
                                          (300, 40, 13001), (40, 700, 40000), (7, 1200, 9000), (2, 3, 131072)])
def test_resize(B, cols, pages):
    rng = np.random.default_rng(B + cols)
    for _ in range(3):
        budget = pages // 2 // B
        lens = rng.integers(0, min(cols, max(budget, 0)) * 64 + 1, B)
        table, refs = pool(rng, lens, cols, pages)
        new = np.clip(lens + rng.integers(-200, 300, B), 0, cols * 64)
        new[rng.random(B) < 0.2] = 0
        check_resize(new, table, refs)


def test_resize_grows_from_nothing_and_frees_all():
    rng = np.random.default_rng(1)
    table, refs = np.full((9, 13), -1, np.int32), np.zeros(200, np.int32)
    t, r, status = check_resize(rng.integers(0, 13 * 64 + 1, 9), table, refs)
    assert status == 0
    t, r, status = check_resize(np.zeros(9, np.int64), t, r)
    assert np.all(t == -1) and np.all(r == 0)


def test_large_pools_that_only_free():
    """Nothing is handed out: the blocks of a cluster end early."""
    rng = np.random.default_rng(11)
    lens = rng.integers(1, 700 * 64, 40) // 2
    table, refs = pool(rng, lens, 700, 40000)
    for new in (np.zeros(40, np.int64), lens // 3, lens):
        for _ in range(3):
            want = check_resize(new, table, refs)
        assert want[2] == 0


def test_resize_hands_out_what_it_gets_back():
    table, refs = np.arange(8, dtype=np.int32).reshape(2, 4), np.ones(8, np.int32)
    t, r, status = check_resize([64, 256], table, refs)
    assert status == 0
    t[0, :] = [0, -1, -1, -1]
    check_resize([0, 256], t, r)
    check_resize([256, 0], t, r)


def test_resize_runs_out_of_pages():
    import paged_mla_decode_09_gb300 as mla

    rng = np.random.default_rng(2)
    table, refs = pool(rng, [100, 0, 500], 12, 11, share=0)
    want = check_resize([768, 768, 768], table, refs)
    assert want[2] == mla.MLA_DEV_NO_PAGES and np.all(want[1] >= 1)


def test_resize_flags():
    import paged_mla_decode_09_gb300 as mla

    table, refs = np.array([[0, 1, -1], [2, -1, -1]], np.int32), np.array([1, 1, 1, 0, 0], np.int32)
    # lengths outside the table are clamped
    t, r, status = resize([1000, -4], table, refs)
    assert status == mla.MLA_DEV_BAD_SEQ_LEN
    assert t.tolist() == [[0, 1, 2], [-1] * 3] and r.tolist() == [1, 1, 1, 0, 0]
    # ids behind the pool count nothing; they stay where they are needed
    bad = table.copy()
    bad[0, 1], bad[1, 0] = 5, 2**31 - 1
    t, r, status = resize([128, 0], bad, refs)
    assert status == mla.MLA_DEV_BAD_PAGE_ID and t.tolist() == [[0, 5, -1], [-1] * 3] and r.tolist() == refs.tolist()
    # a page given back twice, and a count below 0 that was there
    twice, counts = np.array([[0, 1, -1], [0, -1, -1]], np.int32), np.array([1, 1, -3, 0, 1], np.int32)
    t, r, status = resize([0, 0], twice, counts)
    assert status == mla.MLA_DEV_BAD_REFS and r.tolist() == [0, 0, 0, 0, 1]
    # (page 0's count said one row, and one gave it back: it is free, and the lowest)
    t, r, status = resize([192, 0], twice, counts)
    assert t[0].tolist() == [0, 1, 0] and r.tolist() == [1, 1, 0, 0, 1] and status == mla.MLA_DEV_BAD_REFS


def test_resize_of_slices_at_odd_addresses():
    import paged_mla_decode_09_gb300 as mla

    rng = np.random.default_rng(3)
    table, refs = pool(rng, [100, 900, 64], 17, 99, share=0)
    new = [300, 10, 640]
    want = oracle.page_resize_ref(new, table, refs)
    wide, out = torch.full((3, 23), -8, dtype=torch.int32, device="cuda"), torch.full((3, 29), -8, dtype=torch.int32, device="cuda")
    r, ro = torch.zeros(101, dtype=torch.int32, device="cuda"), torch.zeros(102, dtype=torch.int32, device="cuda")
    wide[:, 3:20], r[1:100] = cuda(table), cuda(refs)
    ws = torch.empty(mla.mla_page_resize_workspace_size(3, 17, 99), dtype=torch.uint8, device="cuda")
    mla.mla_page_resize(cuda(np.asarray(new, np.int32)), wide[:, 3:20], r[1:100], out[:, 5:22], ro[3:102], ws)
    assert np.array_equal(out[:, 5:22].cpu().numpy(), want[0]) and np.array_equal(ro[3:].cpu().numpy(), want[1])
    assert torch.all(out[:, :5] == -8) and torch.all(out[:, 22:] == -8) and torch.all(ro[:3] == 0)


def fork_case(rng, lens, src, cols, layers, dtype, spare=None):
    need = sum(-(-int(n) // 64) for n in lens)
    pages = max(1, need + (len(src) + 2 if spare is None else spare))
    table, refs = pool(rng, lens, cols, pages)
    cache = rng.integers(0, 256 if dtype == np.uint8 else 65536, size=(layers, pages, 64, 576)).astype(dtype)
    return np.asarray(src, np.int32), np.asarray(lens, np.int32), table, refs, cache


def fork(src, lens, table, refs, cache, in_place=False):
    import paged_mla_decode_09_gb300 as mla

    t, r = cuda(table), cuda(refs)
    c = cuda(cache.view(np.int16)).view(torch.bfloat16) if cache.dtype == np.uint16 else cuda(cache)
    to, ro = torch.full((len(src), table.shape[1]), -5, dtype=torch.int32, device="cuda"), r if in_place else torch.full_like(r, -5)
    ws = torch.full((mla.mla_page_fork_workspace_size(len(lens), len(src), table.shape[1], len(refs)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    mla.mla_page_fork(cuda(src), cuda(lens), t, r, c, to, ro, ws)
    torch.cuda.synchronize()
    raw = c.view(torch.int16).cpu().numpy().view(np.uint16) if cache.dtype == np.uint16 else c.cpu().numpy()
    assert np.array_equal(t.cpu().numpy(), table)
    return to.cpu().numpy(), ro.cpu().numpy(), raw, mla.mla_query_status(ws)


def check_fork(*case):
    want = oracle.page_fork_ref(*case)
    for in_place in (False, True):
        got = fork(*case, in_place=in_place)
        assert got[3] == want[3]
        for g, w in zip(got[:3], want[:3]):
            assert np.array_equal(g, w), np.argwhere(g != w)[:5].tolist()
    return want


@pytest.mark.parametrize("dtype", [np.uint16, np.uint8])
@pytest.mark.parametrize("lens,children,layers", [([1], 1, 1), ([64], 3, 2), ([0], 2, 1), ([63, 65, 128, 0, 700], 9, 3),
                                                  ([100] * 20, 50, 2), ([37 * k for k in range(30)], 30, 1)])
def test_fork(lens, children, layers, dtype):
    rng = np.random.default_rng(children)
    cols = max(1, max(-(-n // 64) for n in lens)) + 1
    for _ in range(2):
        src = rng.integers(-1, len(lens), children)
        check_fork(*fork_case(rng, lens, src, cols, layers, dtype))


def test_fork_over_many_rows():
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 130, 700)
    check_fork(*fork_case(rng, lens, rng.integers(0, 700, 900), 40, 1, np.uint8))


@pytest.mark.parametrize("spare", [10239 - 72 - 4, 10240 - 72 - 4, 10241 - 72 - 4, 16400])
def test_fork_around_the_size_from_which_a_cluster_does_it(spare):
    rng = np.random.default_rng(spare)
    check_fork(*fork_case(rng, [70, 130], rng.integers(0, 2, 24), 3, 1, np.uint8, spare=spare))


@pytest.mark.parametrize("pages", [16383 - 72, 16384 - 72, 16385 - 72])
def test_resize_around_the_size_from_which_a_cluster_does_it(pages):
    rng = np.random.default_rng(pages)
    lens = rng.integers(0, 193, 24)
    table, refs = pool(rng, lens, 3, pages)
    for _ in range(2):
        check_resize(np.clip(lens + rng.integers(-100, 100, 24), 0, 192), table, refs)


def test_fork_runs_out_of_pages():
    import paged_mla_decode_09_gb300 as mla

    rng = np.random.default_rng(8)
    want = check_fork(*fork_case(rng, [70, 128, 5], [0, 2, 1, 2, 0], 3, 2, np.uint16, spare=2))
    assert want[3] == mla.MLA_DEV_NO_PAGES


def test_fork_flags():
    import paged_mla_decode_09_gb300 as mla

    rng = np.random.default_rng(9)
    src, lens, table, refs, cache = fork_case(rng, [70, 130], [1, 0], 4, 1, np.uint8)
    want = oracle.page_fork_ref([1, -1], lens, table, refs, cache)
    for bad in (2, -2, 2**31 - 1):
        got = fork(np.asarray([1, bad], np.int32), lens, table, refs, cache)
        assert got[3] == mla.MLA_DEV_BAD_INDEX
        assert all(np.array_equal(g, w) for g, w in zip(got[:3], want[:3]))
    for n in (-1, 257):
        bad = lens.copy()
        bad[0] = n
        assert fork(src, bad, table, refs, cache)[3] & mla.MLA_DEV_BAD_SEQ_LEN
    # a full page and a started one with bad ids: -1 in their places, nothing counted or copied
    bad = table.copy()
    bad[0, 0], bad[0, 1] = 10**6, -1
    t, r, c, status = fork(np.asarray([0], np.int32), lens, bad, refs, cache)
    assert status == mla.MLA_DEV_BAD_PAGE_ID and t.tolist() == [[-1] * 4]
    assert np.array_equal(r, refs) and np.array_equal(c, cache)


def test_a_beam_step_keeps_the_pool_whole():
    """Forks, growth and frees in turn, captured: counts are always the tables'."""
    import paged_mla_decode_09_gb300 as mla

    rng = np.random.default_rng(10)
    B, cols, pages, layers = 6, 5, 64, 2
    cache = torch.zeros((layers, pages, 64, 576), dtype=torch.uint8, device="cuda")
    tables = [torch.full((B, cols), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    refs, lens = torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.full((B,), 30, dtype=torch.int32, device="cuda")
    src, zero = torch.arange(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    rws = torch.empty(mla.mla_page_resize_workspace_size(B, cols, pages), dtype=torch.uint8, device="cuda")
    fws = torch.empty(mla.mla_page_fork_workspace_size(B, B, cols, pages), dtype=torch.uint8, device="cuda")
    mla.mla_page_resize(lens, tables[0], refs, tables[0], refs, rws)
    graphs = []
    for k in range(2):  # the graphs share their workspaces
        a, b = tables[k], tables[1 - k]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mla.mla_page_fork(src, lens, a, refs, cache, b, refs, fws)
            mla.mla_page_resize(zero, a, refs, a, refs, rws)   # the old rows end
            lens.copy_(lens[src.long()] + 17)
            mla.mla_page_resize(lens, b, refs, b, refs, rws)
        graphs.append(g)
    ref_t, ref_r, n = tables[0].cpu().numpy(), refs.cpu().numpy(), lens.cpu().numpy()
    ref_c = cache.cpu().numpy()
    for step in range(14):
        s = rng.integers(0, B, B).astype(np.int32)
        src.copy_(torch.from_numpy(s))
        graphs[step % 2].replay()
        torch.cuda.synchronize()
        t2, ref_r, ref_c, st = oracle.page_fork_ref(s, n, ref_t, ref_r, ref_c)
        _, ref_r, st2 = oracle.page_resize_ref([0] * B, ref_t, ref_r)
        n = n[s] + 17
        ref_t, ref_r, st3 = oracle.page_resize_ref(n, t2, ref_r)
        assert st == st2 == st3 == 0
        assert np.array_equal(tables[1 - step % 2].cpu().numpy(), ref_t) and np.array_equal(refs.cpu().numpy(), ref_r)
        assert np.array_equal(np.bincount(ref_t[ref_t >= 0], minlength=pages), ref_r)
        assert torch.all(tables[step % 2] == -1)
