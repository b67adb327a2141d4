"""mla_verify against the float64 oracle: every output is a whole number and
has to be equal.  (The oracle adds up in 64-bit floating point, the kernel in
units of 2^-60; a random number would have to fall within about 2^-40 of a
border for them to differ, a chance of 2^-40 times the entries of a row.)"""
import numpy as np
import pytest

import oracle
import tree_cases as TC

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


def softmax(x):
    e = np.exp(x - x.max(axis=1, keepdims=True))
    return (e / e.sum(axis=1, keepdims=True)).astype(np.float32)


def make(nodes, vocab, drafted, kind="tree", seed=0, sharp=4.0, noise=0.8):
    rng = np.random.default_rng(seed)
    T = max(1, sum(nodes))
    x = sharp * rng.standard_normal((T, vocab))
    target, draft = softmax(x), softmax(x + noise * rng.standard_normal((T, vocab)))
    parents, tokens, at = [], [], 0
    for n in nodes:
        p = ([i - 1 for i in range(n)] if kind == "chain" else [-1] + [0] * (n - 1) if kind == "star"
             else TC.random_tree(rng, n, forest=kind == "forest")) if n else []
        parents += p
        for j, q in enumerate(p):
            row = draft[at + max(q, 0)].astype(np.float64)
            if drafted:
                tokens.append(int(rng.choice(vocab, p=row / row.sum())))
            else:
                tokens.append(int(np.argsort(-row)[sum(q == y for y in p[:j]) % vocab]))
        at += n
    if not parents:
        parents, tokens = [-1], [0]
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    return dict(target=target, draft=draft if drafted else None, tokens=np.asarray(tokens, np.int32),
                parents=np.asarray(parents, np.int32), cu=cu, accept=rng.random(T).astype(np.float32),
                sample=rng.random(len(nodes)).astype(np.float32))


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Run:
    def __init__(self, c, cols):
        self.t = {k: None if v is None else cuda(v) for k, v in c.items()}
        B = len(c["sample"])
        self.path = torch.full((B, cols), -77, dtype=torch.int32, device="cuda")
        self.out, self.num = self.path.clone(), torch.full((B,), -77, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def launch(self, stream=None):
        import paged_mla_decode_09_gb300 as mla

        t = self.t
        mla.mla_verify(t["target"], t["draft"], t["tokens"], t["parents"], t["cu"], t["accept"], t["sample"], self.path,
                       self.out, self.num, self.status, stream)
        return self

    def result(self):
        torch.cuda.synchronize()
        return self.path.cpu().numpy(), self.out.cpu().numpy(), self.num.cpu().numpy(), int(self.status.item())


def check(c, cols, run=None):
    path, out, num, status = (run or Run(c, cols).launch()).result()
    want = oracle.verify_ref(c["target"], c["draft"], c["tokens"], c["parents"], c["cu"], c["accept"], c["sample"], cols)
    assert status == 0
    for name, got, ref in zip(("num", "path", "tokens"), (num, path, out), (want[2], want[0], want[1])):
        assert np.array_equal(got, ref), (name, np.argwhere(got != ref)[:5].tolist())
    return want


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("kind", ["chain", "tree", "star", "forest"])
@pytest.mark.parametrize("vocab", [1, 2, 31, 255, 256, 257, 2047, 5000, 33001])
def test_parity(vocab, kind, drafted):
    nodes = [1, 5, 0, 9, 2, 17] if vocab > 1000 else [1, 5, 0, 9, 2, 33, 4, 4, 4, 4, 8, 8, 8, 70]
    total = 0
    for seed in range(3):
        want = check(make(nodes, vocab, drafted, kind, seed=seed + vocab), cols=max(nodes))
        total += int(want[2].sum())
    assert total > 3 * (len(nodes) - 1) or vocab == 1 or kind == "forest"  # some were accepted


@pytest.mark.parametrize("drafted", [True, False])
def test_largest_trees_and_short_paths(drafted):
    check(make([256, 1, 256], 700, drafted, "chain", seed=1, noise=0.05), cols=256)
    check(make([256, 3], 700, drafted, "star", seed=2, noise=3.0), cols=4)
    for cols in (1, 2, 3, 300):
        check(make([20, 6, 1], 999, drafted, "chain", seed=cols, noise=0.1), cols=cols)


@pytest.mark.parametrize("drafted", [True, False])
def test_large_vocabularies(drafted):
    check(make([4, 3], 131072, drafted, "chain", seed=3), cols=4)
    check(make([3], 1 << 20, drafted, "star", seed=4, noise=2.0), cols=3)


def test_many_rejected_siblings():
    """Drafts far from the target: several sums per request."""
    c = make([40] * 12, 3000, True, "star", seed=6, noise=6.0)
    check(c, cols=5)
    c = make([12] * 9, 400, True, "star", seed=7, noise=9.0, sharp=1.0)
    c["accept"][:] = 0.999
    check(c, cols=5)


def test_same_token_twice_and_exact_rows():
    """Rows of few bits, where draft and target are equal or disjoint."""
    rng = np.random.default_rng(9)
    T, V = 6 * 40, 8
    eighths = rng.multinomial(8, np.ones(V) / V, size=T).astype(np.float32) / 8
    draft = eighths.copy()
    draft[::3] = np.roll(eighths[::3], 1, axis=1)
    for drafted in (True, False):
        c = dict(target=eighths, draft=draft if drafted else None, tokens=rng.integers(0, V, T).astype(np.int32),
                 parents=np.tile([-1, 0, 0, 0, 1, 1], 40).astype(np.int32), cu=np.arange(41, dtype=np.int32) * 6,
                 accept=(rng.integers(0, 16, T) / 16).astype(np.float32),
                 sample=(rng.integers(0, 16, 40) / 16).astype(np.float32))
        check(c, cols=4)


def test_random_numbers_at_their_ends():
    c = make([5, 5, 5, 5], 1000, True, "chain", seed=10)
    for a, s in ((0.0, 0.0), (np.nextafter(np.float32(1), np.float32(0)),) * 2, (0.0, np.float32(1e-30))):
        c["accept"][:], c["sample"][:] = a, s
        check(c, cols=5)
    # outside [0, 1): taken as the nearest inside
    c["accept"][:] = 0.5
    c["sample"][:] = [1.0, np.inf, -3.0, np.nan]
    got = Run(c, 5).launch().result()
    c["sample"][:] = [np.nextafter(np.float32(1), np.float32(0))] * 2 + [0.0, 0.0]
    want = Run(c, 5).launch().result()
    assert all(np.array_equal(x, y) for x, y in zip(got[:3], want[:3])) and got[3] == 0


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("kind", ["chain", "star"])
def test_acceptance_numbers_outside_their_range(kind, drafted):
    """Taken as the nearest inside, a NaN as 0, at a node's first child and at
    later ones; above all a token that the target gives nothing is not accepted."""
    c = make([6] * 40, 50, drafted, kind, seed=14, noise=2.0)
    rng = np.random.default_rng(15)
    odd = np.asarray([-1.0, -np.inf, np.nan, 1.0, 7.0, np.inf, -0.0, -1e-30], np.float32)
    inside = np.asarray([0, 0, 0, *[np.nextafter(np.float32(1), np.float32(0))] * 3, 0, 0], np.float32)
    pick = rng.integers(0, 8, len(c["accept"]))
    c["target"][np.arange(1, 240), c["tokens"][1:]] = 0.0  # some rows lose a token's weight
    c["target"][0::2, :25] = 0.0
    clean = dict(c, accept=inside[pick])
    want = oracle.verify_ref(clean["target"], clean["draft"], clean["tokens"], clean["parents"], clean["cu"],
                             clean["accept"], clean["sample"], 6)
    path, out, num, status = Run(dict(c, accept=odd[pick]), 6).launch().result()
    assert status == 0
    assert np.array_equal(path, want[0]) and np.array_equal(num, want[2]) and np.array_equal(out, want[1])
    # one request whose draft has no weight at all: rejected whatever its number
    p = np.zeros((2, 8), np.float32)
    p[:, 3] = 1.0
    q = np.full((2, 8), 0.125, np.float32)
    one = dict(target=p, draft=q if drafted else None, tokens=np.array([0, 5], np.int32),
               parents=np.array([-1, 0], np.int32), cu=np.array([0, 2], np.int32), sample=np.array([0.5], np.float32))
    for u in odd:
        path, out, num, status = Run(dict(one, accept=np.asarray([0, u], np.float32)), 2).launch().result()
        assert status == 0 and num.tolist() == [1] and out.tolist() == [[3, -1]], u


def test_odd_values_in_rows():
    """NaN and negative entries count as nothing, entries above 1 as 1; a row
    with nothing in it raises a flag."""
    import paged_mla_decode_09_gb300 as mla

    c = make([1, 1, 1], 600, False, seed=11)
    clean = {k: None if v is None else v.copy() for k, v in c.items()}
    c["target"][0, 7::9] = np.nan
    c["target"][1, 3::5] = -np.inf
    clean["target"][0, 7::9] = 0
    clean["target"][1, 3::5] = 0
    c["target"][2, :] = 0
    c["target"][2, 500] = np.inf
    clean["target"][2, :] = 0
    clean["target"][2, 500] = 1
    path, out, num, status = Run(c, 2).launch().result()
    want = oracle.verify_ref(clean["target"], None, c["tokens"], c["parents"], c["cu"], c["accept"], c["sample"], 2)
    assert status == 0 and np.array_equal(out, want[1]) and np.array_equal(num, want[2])
    c["target"][1, :] = 0
    path, out, num, status = Run(c, 2).launch().result()
    assert status == mla.MLA_DEV_BAD_PROBS and out[1].tolist() == [-1, -1] and num[1] == 1 and out[0, 0] == want[1][0, 0]
    # a rejection that leaves nothing falls back on the node's own row
    p = np.zeros((2, 50), np.float32)
    p[:, 5] = 1.0
    c = dict(target=p, draft=p.copy(), tokens=np.array([0, 9], np.int32), parents=np.array([-1, 0], np.int32),
             cu=np.array([0, 2], np.int32), accept=np.array([0, 0.5], np.float32), sample=np.array([0.3], np.float32))
    path, out, num, status = Run(c, 2).launch().result()
    assert status == 0 and num.tolist() == [1] and out.tolist() == [[5, -1]] and path.tolist() == [[0, -1]]


def test_bad_nodes_and_offsets():
    import paged_mla_decode_09_gb300 as mla

    c = make([4, 6, 3], 500, True, "tree", seed=12)
    for key, at, value, flag in (("tokens", 5, 500, mla.MLA_DEV_BAD_INDEX), ("tokens", 5, -1, mla.MLA_DEV_BAD_INDEX),
                                 ("parents", 5, 1, mla.MLA_DEV_BAD_TREE), ("parents", 5, -5, mla.MLA_DEV_BAD_TREE)):
        d = {k: v.copy() for k, v in c.items()}
        d[key][at] = value
        path, out, num, status = Run(d, 6).launch().result()
        assert status == flag
        gone = {k: v.copy() for k, v in c.items()}  # as if node 1 of request 1 were not there
        gone["parents"][5] = -1
        want = oracle.verify_ref(gone["target"], gone["draft"], gone["tokens"], gone["parents"], gone["cu"],
                                 gone["accept"], gone["sample"], 6)
        assert np.array_equal(path, want[0]) and np.array_equal(out, want[1]) and np.array_equal(num, want[2])
    want = oracle.verify_ref(c["target"], c["draft"], c["tokens"], c["parents"], c["cu"], c["accept"], c["sample"], 6)
    for cu in ([0, 4, 3, 13], [1, 4, 10, 13], [0, 4, 10, 14], [0, 4, -10, 2**31 - 1]):
        d = dict(c, cu=np.asarray(cu, np.int32))
        path, out, num, status = Run(d, 6).launch().result()
        assert status & mla.MLA_DEV_BAD_QUERY_RANGE
        if cu[0] == 0:
            assert np.array_equal(path[0], want[0][0]) and out[0].tolist() == want[1][0].tolist()
        else:
            assert num[0] == 0 and np.all(path[0] == -1) and np.all(out[0] == -1)
    d = make([257, 3], 40, True, "chain", seed=13)
    path, out, num, status = Run(d, 6).launch().result()
    assert status == mla.MLA_DEV_BAD_TREE and num[0] == 0 and np.all(out[0] == -1) and num[1] >= 1


def test_node_0_stays_whatever_its_parent():
    import paged_mla_decode_09_gb300 as mla

    c = make([4, 6, 3], 500, True, "tree", seed=12)
    want = check(c, 6)
    for value in (0, 3, -2, 2**31 - 1):
        d = dict(c, parents=c["parents"].copy())
        d["parents"][4] = value
        path, out, num, status = Run(d, 6).launch().result()
        assert status == mla.MLA_DEV_BAD_TREE
        assert np.array_equal(path, want[0]) and np.array_equal(out, want[1]) and np.array_equal(num, want[2])


@pytest.mark.parametrize("pad", [1, 2, 3, 4, 7])
def test_strides_and_alignment(pad):
    """Rows of a wider tensor, at any offset of four bytes."""
    c = make([5, 9, 1], 1003, True, "tree", seed=pad)
    r = Run(c, 9)
    for k in ("target", "draft"):
        wide = torch.full((r.t[k].shape[0], 1003 + pad + 2), float("nan"), device="cuda")
        wide[:, pad:pad + 1003] = r.t[k]
        r.t[k] = wide[:, pad:pad + 1003]
    check(c, 9, r.launch())


def test_streams_and_captures():
    cs = [make([5] * 7, 3001, True, "chain", seed=20), make([9] * 7, 3001, True, "tree", seed=21)]
    runs = [Run(c, 9) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(4):
        for r, s in zip(runs, streams):
            r.launch(s)
    for c, r in zip(cs, runs):
        check(c, 9, r)
    r = runs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.launch()
    for seed in (30, 31):  # a replay reads its inputs anew
        c = make([5] * 7, 3001, True, "chain", seed=seed)
        for k, v in c.items():
            r.t[k].copy_(cuda(v))
        g.replay()
        check(c, 9, r)
