"""Whole speculative steps, as a serving loop runs them: pages for the trees,
the rotated rows' cache write and the trees' attention in every layer,
verification, the accepted rows' move, pages given back, and a fork.  What a
step leaves in the cache, and what it attended to, is compared with a request
that only ever had the accepted tokens."""
from types import SimpleNamespace

import numpy as np
import pytest

import oracle
import tree_cases as TC

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LAYERS, HEADS, VOCAB, PAGES, COLS = 2, 8, 331, 40, 6
SCALE = 0.1


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


class Server:
    """Buffers of a serving loop over B requests with trees of fixed sizes."""

    def __init__(self, nodes, start, kv, seed=0):
        import paged_mla_decode_09_gb300 as mla

        self.nodes, self.kv, self.B, self.T = nodes, kv, len(nodes), sum(nodes)
        self.rng = np.random.default_rng(seed)
        self.plan = mla.mla_rope_plan(64, interleaved=True)
        dt = torch.bfloat16 if kv == "bf16" else torch.uint8
        self.kv_scale = 1.0 if kv == "bf16" else 0.02
        self.cache = torch.zeros((LAYERS, PAGES, 64, 576), dtype=dt, device="cuda")
        self.table = torch.full((self.B, COLS), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.lens = [i32(start), i32(start)]  # committed tokens, before and after a step
        self.n, self.cu = i32(nodes), i32(np.concatenate([[0], np.cumsum(nodes)]))
        self.total = torch.zeros(self.B, dtype=torch.int32, device="cuda")
        z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        self.q_nope, self.q_raw = z(LAYERS, self.T, HEADS, 512, t=bf), z(LAYERS, self.T, HEADS, 64, t=bf)
        self.q_pe, self.rows = z(LAYERS, self.T, HEADS, 64, t=bf), z(LAYERS, self.T, 576, t=bf)
        self.out, self.lse = z(LAYERS, self.T, HEADS, 512, t=bf), z(LAYERS, self.T, HEADS, t=torch.float32)
        self.parents, self.depth, self.positions, self.tokens = z(self.T), z(self.T), z(self.T), z(self.T)
        self.target, self.draft = z(self.T, VOCAB, t=torch.float32), z(self.T, VOCAB, t=torch.float32)
        self.accept, self.sample = z(self.T, t=torch.float32), z(self.B, t=torch.float32)
        self.path, self.next, self.num = z(self.B, max(nodes)), z(self.B, max(nodes)), z(self.B)
        self.status = z(1)
        self.head = torch.randn(HEADS * 512, VOCAB, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        self.owner = i32(np.repeat(np.arange(self.B), nodes)).long()
        dims = mla.make_prefill_dims(self.q_nope[0], self.cache[0], self.table, self.total)
        self.ws = torch.zeros(mla.mla_decode_tree_workspace_size(dims), dtype=torch.uint8, device="cuda")
        self.pws = torch.zeros(mla.mla_page_resize_workspace_size(self.B, COLS, PAGES), dtype=torch.uint8, device="cuda")
        # the tokens that are there at the beginning
        mla.mla_page_resize(self.lens[0], self.table, self.refs, self.table, self.refs, self.pws)
        rows = torch.randn((LAYERS, sum(start), 576), device="cuda").to(bf)
        q = torch.zeros((sum(start), 1, 64), dtype=bf, device="cuda")
        cu = i32(np.concatenate([[0], np.cumsum(start)]))
        for k in range(LAYERS):
            mla.mla_rope_pack(self.plan, q, rows[k], None, self.table, self.lens[0], cu, self.kv_scale, q,
                              self.cache[k], self.status)

    def draw(self):
        """New trees, rows, queries and random numbers."""
        trees = [TC.random_tree(self.rng, n, near=3) for n in self.nodes]
        depth = []
        for t in trees:
            d = []
            for p in t:
                d.append(0 if p < 0 else d[p] + 1)
            depth += d
        self.parents.copy_(i32(sum(trees, [])))
        self.depth.copy_(i32(depth))
        for t in (self.q_nope, self.q_raw, self.rows):
            t.copy_(torch.from_numpy(self.rng.standard_normal(t.shape).astype(np.float32)))
        x = self.rng.standard_normal((self.T, VOCAB)) * 3
        e = np.exp(x - x.max(axis=1, keepdims=True))
        e /= e.sum(axis=1, keepdims=True)
        self.draft.copy_(torch.from_numpy(e.astype(np.float32)))
        at, tokens = 0, []
        for t in trees:
            tokens += [0 if p < 0 else int(self.rng.choice(VOCAB, p=e[at + p])) for p in t]
            at += len(t)
        self.tokens.copy_(i32(tokens))
        self.accept.copy_(torch.from_numpy(self.rng.random(self.T).astype(np.float32)))
        self.sample.copy_(torch.from_numpy(self.rng.random(self.B).astype(np.float32)))

    def step(self, k=0):
        """A step from lens[k] to lens[1 - k]; nothing here waits for the GPU."""
        import paged_mla_decode_09_gb300 as mla

        before, after = self.lens[k], self.lens[1 - k]
        torch.add(before, self.n, out=self.total)
        torch.add(before[self.owner], self.depth, out=self.positions)
        mla.mla_page_resize(self.total, self.table, self.refs, self.table, self.refs, self.pws)
        for layer in range(LAYERS):
            mla.mla_rope_pack(self.plan, self.q_raw[layer], self.rows[layer], self.positions, self.table, self.total,
                              self.cu, self.kv_scale, self.q_pe[layer], self.cache[layer], self.status)
            mla.mla_decode_tree(self.q_nope[layer], self.q_pe[layer], self.cache[layer], self.table, self.total,
                                self.cu, self.parents, SCALE, self.kv_scale, self.out[layer], self.lse[layer], self.ws)
        # a head whose distribution is near the draft's
        logits = torch.log(self.draft) + 0.02 * (self.out[-1].float().view(self.T, -1) @ self.head)
        self.target.copy_(torch.softmax(logits, dim=1))
        mla.mla_verify(self.target, self.draft, self.tokens, self.parents, self.cu, self.accept, self.sample, self.path,
                       self.next, self.num, self.status)
        mla.mla_tree_commit(self.cache, self.table, self.total, self.cu, self.path, self.num, after, self.status)
        mla.mla_page_resize(after, self.table, self.refs, self.table, self.refs, self.pws)

    def bits(self, t):
        return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()

    def request_rows(self, b, n):
        """The first n cached rows of a request, every layer."""
        pages = self.table[b, :-(-n // 64)].long()
        return self.bits(self.cache[:, pages].reshape(LAYERS, -1, 576)[:, :n].contiguous())

    def check_pool(self):
        table = self.table.cpu().numpy()
        assert np.array_equal(np.bincount(table[table >= 0], minlength=PAGES), self.refs.cpu().numpy())


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_steps_leave_what_the_accepted_tokens_alone_would(kv):
    import paged_mla_decode_09_gb300 as mla

    s = Server([9, 1, 17], [60, 5, 130], kv)
    rows = [s.request_rows(b, int(s.lens[0][b])) for b in range(3)]
    moved = 0
    for k in range(6):
        s.draw()
        s.step(k % 2)
        torch.cuda.synchronize()
        assert s.status.item() == 0 and mla.mla_query_status(s.ws) == 0 and mla.mla_query_status(s.pws) == 0
        before, after = s.lens[k % 2].tolist(), s.lens[1 - k % 2].tolist()
        num, path = s.num.tolist(), s.path.tolist()
        want = oracle.verify_ref(s.target.cpu().numpy(), s.draft.cpu().numpy(), s.tokens.tolist(), s.parents.tolist(),
                                 s.cu.tolist(), s.accept.tolist(), s.sample.tolist(), max(s.nodes))
        assert np.array_equal(s.path.cpu().numpy(), want[0]) and np.array_equal(s.next.cpu().numpy(), want[1])
        s.check_pool()
        for b in range(3):
            assert after[b] == before[b] + num[b] and num[b] >= 1
            moved += any(path[b][j] != j for j in range(num[b]))
            # the rows of before are as they were; the accepted ones' are theirs, turned by their positions
            new = s.request_rows(b, after[b])
            assert np.array_equal(new[:, :before[b]], rows[b])
            rows[b] = new
            at = s.cu.tolist()[b]
            fresh = torch.zeros((LAYERS, 1, 64, 576), dtype=s.cache.dtype, device="cuda")
            nodes = [at + j for j in path[b][:num[b]]]
            q = torch.zeros((num[b], 1, 64), dtype=torch.bfloat16, device="cuda")
            for layer in range(LAYERS):
                mla.mla_rope_pack(s.plan, q, s.rows[layer][nodes].contiguous(), i32(range(before[b], after[b])), i32([[0]]),
                                  i32([num[b]]), i32([0, num[b]]), s.kv_scale, q, fresh[layer], s.status)
            assert np.array_equal(s.bits(fresh)[:, 0, :num[b]], new[:, before[b]:])
            # what an accepted node attended to is what a request of its tokens alone has
            for layer in range(LAYERS):
                c = SimpleNamespace(q_nope=s.bits(s.q_nope[layer][nodes].contiguous()),
                                    q_pe=s.bits(s.q_pe[layer][nodes].contiguous()), kv_cache=s.bits(s.cache[layer]),
                                    page_table=s.table.cpu().numpy()[b:b + 1], kv_dtype=kv, kv_scale=s.kv_scale, scale=SCALE,
                                    cu=[0])
                for j, node in enumerate(nodes):
                    ref, lse, to, tl = TC.error_bounds(c, 0, j, np.arange(before[b] + j + 1))
                    assert np.all(np.abs(s.out[layer][node].double().cpu().numpy() - ref) <= to)
                    assert np.all(np.abs(s.lse[layer][node].double().cpu().numpy() - lse) <= tl)
    assert moved > 0  # some accepted rows were not in their places


def test_a_captured_step_is_the_eager_one():
    """Two graphs, one for each direction of the lengths' two buffers."""
    a, b = Server([9, 4, 17], [60, 5, 130], "bf16", seed=4), Server([9, 4, 17], [60, 5, 130], "bf16", seed=4)
    b.cache.copy_(a.cache)
    graphs = []
    saved = [t.clone() for t in (b.cache, b.table, b.refs, *b.lens)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.draw()
        b.step(0)
    torch.cuda.current_stream().wait_stream(side)
    b.rng = np.random.default_rng(4)
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.step(k)
        graphs.append(g)
    for t, v in zip((b.cache, b.table, b.refs, *b.lens), saved):
        t.copy_(v)
    for k in range(5):
        a.draw()
        b.draw()
        a.step(k % 2)
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        for x, y in ((a.out, b.out), (a.next, b.next), (a.num, b.num), (a.lens[1 - k % 2], b.lens[1 - k % 2]),
                     (a.table, b.table), (a.refs, b.refs)):
            assert torch.equal(x, y)
        # rows that are in use (a tree's rejected rows stay behind the length in both)
        for r in range(3):
            n = int(a.lens[1 - k % 2][r])
            assert np.array_equal(a.request_rows(r, n), b.request_rows(r, n))


def test_forked_requests_go_on_apart():
    """Two samples of one request share its full pages and differ behind them."""
    import paged_mla_decode_09_gb300 as mla

    s = Server([5, 5], [100, 20], "bf16", seed=6)
    s.draw()
    s.step(0)
    n = int(s.lens[1][0])
    table = torch.full_like(s.table, -1)
    fws = torch.zeros(mla.mla_page_fork_workspace_size(2, 2, COLS, PAGES), dtype=torch.uint8, device="cuda")
    mla.mla_page_fork(i32([0, 0]), s.lens[1], s.table, s.refs, s.cache, table, s.refs, fws)
    mla.mla_page_resize(i32([0, 0]), s.table, s.refs, s.table, s.refs, s.pws)  # the old rows end
    whole = None
    s.table.copy_(table)
    s.check_pool()
    whole = [s.request_rows(b, n) for b in range(2)]
    assert np.array_equal(whole[0], whole[1])
    s.lens[1].fill_(n)
    s.draw()
    s.step(1)
    torch.cuda.synchronize()
    s.check_pool()
    assert s.status.item() == 0 and mla.mla_query_status(fws) == 0
    t = s.table.cpu().numpy()
    assert np.array_equal(t[0, :n // 64], t[1, :n // 64]) and t[0, n // 64] != t[1, n // 64]
    for b in range(2):
        assert np.array_equal(s.request_rows(b, n), whole[b])
