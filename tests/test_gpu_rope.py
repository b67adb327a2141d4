"""mla_rope_pack against the float64 oracle, value by value.

Bounds: an angle in half turns is rounded to fp32 (at most 2^-25, times pi in
radians) after its exact product; a frequency holds 2^-52 of itself, which at a
position p costs p f 2^-51; sine and cosine are off by at most 2^-22 (2 units in
the last place), the amplitude's product by 2^-24; the two products and their
sum by 2^-23 of |a| + |b|.  Then one rounding to bf16 (2^-8 of the value, which
counts half a step twice over) or to e4m3 (2^-4, and half the step of the least
binade, 2^-10 codes, with the saturation at 448)."""
import math

import numpy as np
import pytest

import oracle
import tree_cases as TC
from paged_mla_decode_09_gb300 import workloads as W

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


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).cuda()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    def __init__(self, new, total, heads, kv="bf16", seed=0, positions=None, extra=0):
        rng = np.random.default_rng(seed)
        self.new, self.kv, self.heads = new, kv, heads
        self.T = T = sum(new) + extra
        self.lens, self.cu = np.asarray(total, np.int32), np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        width = max(1, max(-(-t // 64) for t in total))
        self.table, used = np.full((len(new), width), -1, np.int32), []
        for b, (m, n) in enumerate(zip(new, total)):  # only the pages that receive a row
            if m:
                used += [(b, c) for c in range((n - m) // 64, -(-n // 64))]
        ids = rng.permutation(len(used) + 2)
        for (b, c), i in zip(used, ids):
            self.table[b, c] = i
        self.cache = rng.integers(0, 120, (len(used) + 2, 64, 576)).astype(np.uint8 if kv == "e4m3" else np.uint16)
        self.q = W.f32_to_bf16_bits(rng.standard_normal((T, heads, 64)).astype(np.float32))
        self.rows = W.f32_to_bf16_bits(rng.standard_normal((T, 576)).astype(np.float32))
        self.kv_scale = 0.011 if kv == "e4m3" else 1.0
        first = np.concatenate([np.arange(n - m, n) for m, n in zip(new, total)] + [np.zeros(extra, np.int64)])
        self.slots = positions is None
        self.positions = (first if positions is None else np.asarray(positions)).astype(np.int32)

    def run(self, plan, in_place=False, q=None, rows=None, status=0):
        import paged_mla_decode_09_gb300 as mla

        q = bf16(self.q) if q is None else q
        rows = bf16(self.rows) if rows is None else rows
        out = q if in_place else torch.full((self.T, self.heads, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        cache = cuda(self.cache) if self.kv == "e4m3" else bf16(self.cache)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.mla_rope_pack(plan, q, rows, None if self.slots else cuda(self.positions), cuda(self.table), cuda(self.lens),
                          cuda(self.cu), self.kv_scale, out, cache, st)
        torch.cuda.synchronize()
        assert st.item() == status
        return bits(out), (cache.cpu().numpy() if self.kv == "e4m3" else bits(cache))

    def check(self, plan, freq, interleaved, amplitude=1.0, got=None, requests=None):
        out, cache = got if got is not None else self.run(plan)
        n = int(self.cu[-1])
        pos = self.positions[:n]
        x = oracle.bf16_bits_to_f64(self.q[:n])
        k = oracle.bf16_bits_to_f64(self.rows[:n])
        r = 2 * len(freq)

        def rotated(v):
            ref = oracle.rotate_ref(v, pos, freq, interleaved, amplitude)
            i = np.arange(r // 2)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
            big = np.zeros_like(v)
            big[..., a] = big[..., b] = np.abs(v[..., a]) + np.abs(v[..., b])
            err = np.abs(pos)[:, None] * np.asarray(freq)[None] * 2.0**-51 + math.pi * 2.0**-25 + 2.0**-22 + 2.0**-24 + 2.0**-23
            wide = np.zeros((n, 64))
            wide[:, a] = wide[:, b] = err
            return ref, amplitude * big * wide.reshape((n,) + (1,) * (v.ndim - 2) + (64,))

        ref, err = rotated(x)
        keep = np.ones(n, bool)
        if requests is not None:
            keep[:] = False
            for b in requests:
                keep[self.cu[b]:self.cu[b + 1]] = True
        got_q = oracle.bf16_bits_to_f64(out[:n])
        assert np.all(np.abs(got_q - ref)[keep] <= (2.0**-8 * np.abs(ref) + err * 1.01)[keep])
        assert np.array_equal(out[:n][..., r:][keep], self.q[:n][..., r:][keep])  # what passes, passes unchanged
        ref_k, err_k = rotated(k[:, 512:])
        untouched = np.ones(self.cache.shape[:2], bool)
        for t, (page, row) in enumerate(oracle.new_slots(self.table, self.lens, self.cu)):
            if not keep[t] or page < 0:
                continue
            untouched[page, row] = False
            have = cache[page, row]
            if self.kv == "bf16":
                assert np.array_equal(have[:512], self.rows[t, :512]) and np.array_equal(have[512 + r:], self.rows[t, 512 + r:])
                assert np.all(np.abs(oracle.bf16_bits_to_f64(have[512:]) - ref_k[t]) <= 2.0**-8 * np.abs(ref_k[t]) + err_k[t] * 1.01)
            else:
                scale = np.float64(np.float32(self.kv_scale))
                codes = oracle.e4m3_encode(k[t] / scale)
                assert np.array_equal(have[:512], codes[:512]) and np.array_equal(have[512 + r:], codes[512 + r:])
                want = np.clip(ref_k[t] / scale, -448.0, 448.0)
                val = oracle.e4m3_to_f64(have[512:])
                assert np.all(np.abs(val - want) <= np.maximum(2.0**-4 * np.abs(want), 2.0**-10) + err_k[t] * 1.1 / scale)
        assert np.array_equal(cache[untouched], self.cache[untouched])
        return out, cache


def plan_of(dim, interleaved, amplitude=1.0, **kw):
    import paged_mla_decode_09_gb300 as mla

    freq = oracle.rope_frequencies_ref(dim, **{"base": 10000.0, **kw})
    return mla.mla_rope_plan(dim, interleaved=interleaved, amplitude=amplitude, **kw), freq


SHAPES = {
    "one": dict(new=[1], total=[1], heads=1),
    "one_later": dict(new=[1], total=[65], heads=16),
    "page_edges": dict(new=[1, 63, 64, 65], total=[64, 63, 128, 129], heads=4),
    "odd_heads_no_tokens": dict(new=[0, 5, 0, 30, 0], total=[70, 200, 1, 500, 0], heads=20),
    "wide": dict(new=[3, 17], total=[130, 1000], heads=128),
    "many_requests": dict(new=[1 + k % 3 for k in range(700)], total=[3 + k for k in range(700)], heads=2),
    "rows_behind": dict(new=[9, 3], total=[100, 64], heads=16, extra=5),
    "prompt": dict(new=[700], total=[800], heads=24),
    "very_wide": dict(new=[2], total=[2], heads=1000),
}


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("name", list(SHAPES))
def test_parity(name, interleaved, kv):
    plan, freq = plan_of(64, interleaved)
    c = Case(kv=kv, seed=len(name), **SHAPES[name])
    out, _ = c.check(plan, freq, interleaved)
    n = int(c.cu[-1])
    assert np.all(oracle.bf16_bits_to_f64(out[n:]) == 7.0)  # tokens behind the last request


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dim", [16, 32, 48])
def test_a_part_of_the_head(dim, interleaved, kv):
    plan, freq = plan_of(dim, interleaved)
    Case([7, 2], [80, 300], 5, kv=kv, seed=dim).check(plan, freq, interleaved)


@pytest.mark.parametrize("interleaved", [True, False])
def test_scaled_and_far(interleaved):
    kw = dict(factor=40.0, original_len=4096)
    plan, freq = plan_of(64, interleaved, amplitude=1.3689, **kw)
    pos = [0, 1, 4095, 4096, 163839, 10**6, 2**31 - 1, -1, -12345, 77777]
    Case([10], [70], 3, seed=1, positions=pos).check(plan, freq, interleaved, 1.3689)
    plan, freq = plan_of(64, interleaved, factor=8.0)
    Case([10], [70], 3, kv="e4m3", seed=1, positions=pos).check(plan, freq, interleaved)


def test_nodes_of_one_depth_turn_alike():
    rng = np.random.default_rng(3)
    parents = TC.random_tree(rng, 20)
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    plan, freq = plan_of(64, True)
    Case([20], [90], 4, seed=4, positions=70 + np.asarray(depth)).check(plan, freq, True)


def test_in_place_strided_and_repeated():
    plan, freq = plan_of(64, False)
    c = Case([40, 9], [100, 64], 12, seed=5)
    out, cache = c.check(plan, freq, False)
    again = c.run(plan, in_place=True)
    assert np.array_equal(again[0], out) and np.array_equal(again[1], cache)
    # queries and rows that are slices of wider tensors
    q = torch.zeros((49, 12, 192), dtype=torch.bfloat16, device="cuda")
    q[..., 128:] = bf16(c.q)
    rows = torch.zeros((49, 600), dtype=torch.bfloat16, device="cuda")
    rows[:, 8:584] = bf16(c.rows)
    again = c.run(plan, q=q[..., 128:], rows=rows[:, 8:584])
    assert np.array_equal(again[0], out) and np.array_equal(again[1], cache)
    q = torch.zeros((12, 49, 64), dtype=torch.bfloat16, device="cuda")
    q.copy_(bf16(c.q).transpose(0, 1))
    again = c.run(plan, q=q.transpose(0, 1))
    assert np.array_equal(again[0], out) and np.array_equal(again[1], cache)


@pytest.mark.parametrize("slots", [True, False])
def test_flags(slots):
    import paged_mla_decode_09_gb300 as mla

    plan, freq = plan_of(64, True)

    def case():
        c = Case([3, 5, 2], [100, 200, 90], 4, seed=6)
        c.slots = slots
        return c

    c = case()
    c.lens[1] = 4  # fewer cached tokens than new ones: left out
    good = case()
    got = c.run(plan, status=mla.MLA_DEV_BAD_SEQ_LEN)
    good.check(plan, freq, True, got=(got[0], _without(good, got[1], 1)), requests=[0, 2])
    assert np.all(oracle.bf16_bits_to_f64(got[0][3:8]) == 7.0)
    c = case()
    c.lens[1] = 10**6
    got = c.run(plan, status=mla.MLA_DEV_BAD_SEQ_LEN)
    assert np.all(oracle.bf16_bits_to_f64(got[0][3:8]) == 7.0)
    c = case()
    c.table[1, 3] = 10**6  # the rows are not written, the queries are
    got = c.run(plan, status=mla.MLA_DEV_BAD_PAGE_ID)
    c.table[1, 3] = -1
    c.check(plan, freq, True, got=got)
    for cu in ([0, 3, 2, 10], [0, 3, 8, 11], [1, 3, 8, 10], [0, -5, 8, 10]):
        c = case()
        c.cu = np.asarray(cu, np.int32)
        c.run(plan, status=mla.MLA_DEV_BAD_QUERY_RANGE)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("slots", [True, False])
@pytest.mark.parametrize("cu,owners", [([0, 3, 2, 10], [0, 0, 2, 2, 2, 2, 2, 2, 2, 2]), ([0, 9, 1, 4], [0, 2, 2, 2] + [0] * 5 + [None]),
                                       ([0, 3, 8, 11], [0, 0, 0, 1, 1, 1, 1, 1, None, None]),
                                       ([1, 3, 8, 10], [None] * 3 + [1] * 5 + [2] * 2), ([0, -5, 8, 10], [None] * 8 + [2, 2])])
def test_bad_offsets_leave_the_other_requests_right(cu, owners, slots, kv):
    """A token that two requests name is the last one's; a request with a bad
    offset is left out; everything else is as it would be without them."""
    import paged_mla_decode_09_gb300 as mla

    plan, freq = plan_of(64, True)
    c = Case([3, 5, 2], [100, 200, 90], 4, kv=kv, seed=6)
    c.table = np.arange(12, dtype=np.int32).reshape(3, 4)
    c.cache = np.random.default_rng(8).integers(0, 120, (12, 64, 576)).astype(c.cache.dtype)
    c.cu, c.slots = np.asarray(cu, np.int32), slots
    out, cache = c.run(plan, status=mla.MLA_DEV_BAD_QUERY_RANGE)
    # the same with a request for each token, whose length puts it where its owner does
    one = Case([3, 5, 2], [100, 200, 90], 4, kv=kv, seed=6)
    one.cache, one.slots = c.cache, slots
    kept = [t for t in range(10) if owners[t] is not None]
    one.table = np.stack([c.table[owners[t]] for t in kept])
    one.lens = np.asarray([c.lens[owners[t]] - c.cu[owners[t] + 1] + t + 1 for t in kept], np.int32)
    one.cu = np.arange(len(kept) + 1, dtype=np.int32)
    one.q, one.rows, one.T, one.positions = c.q[kept], c.rows[kept], len(kept), c.positions[kept]
    want, rows = one.run(plan)
    assert np.array_equal(out[kept], want) and np.array_equal(cache, rows)
    gone = [t for t in range(10) if owners[t] is None]
    assert np.all(oracle.bf16_bits_to_f64(out[gone]) == 7.0)


def _without(c, cache, b):
    """The cache, after checking that request b's rows are as they were."""
    n = int(c.cu[b + 1] - c.cu[b])
    for t in range(int(c.lens[b]) - n, int(c.lens[b])):
        assert np.array_equal(cache[c.table[b, t // 64], t % 64], c.cache[c.table[b, t // 64], t % 64])
    return cache


def test_captured_and_on_streams():
    import paged_mla_decode_09_gb300 as mla

    plan, freq = plan_of(64, True)
    c = Case([6, 3], [70, 90], 8, seed=7, positions=np.arange(9))
    q, rows, pos = bf16(c.q), bf16(c.rows), cuda(c.positions)
    out, cache = torch.zeros_like(q), bf16(c.cache)
    rest = cuda(c.table), cuda(c.lens), cuda(c.cu)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_rope_pack(plan, q, rows, pos, *rest, 1.0, out, cache, st)
    plan.turn[0] = 0  # the plan was read by the call
    for first in (0, 5000):
        c.positions = (first + np.arange(9)).astype(np.int32)
        pos.copy_(cuda(c.positions))
        g.replay()
        torch.cuda.synchronize()
        c.check(None, freq, True, got=(bits(out), bits(cache)))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    mla.mla_rope_pack(plan_of(64, True)[0], q, rows, pos, *rest, 1.0, out, cache, st, stream=s)
    torch.cuda.synchronize()
    c.check(None, freq, True, got=(bits(out), bits(cache)))
    assert st.item() == 0
