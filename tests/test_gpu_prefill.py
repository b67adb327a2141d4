"""GPU parity of mla_prefill and mla_decode_window against the float64 oracle,
element by element with the bounds of chunk_cases.error_bounds: ragged chunks,
requests without queries, odd head counts, windows and sinks across page
borders, contexts cut into many pieces, both cache types."""
import numpy as np
import pytest

import chunk_cases as K
import oracle
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


SENTINEL = 7.0


class Run:
    """Device copies of a case, with outputs and a workspace full of garbage."""

    def __init__(self, c):
        import paged_mla_decode_09_gb300 as mla

        self.c = c
        self.qn, self.qp = K.to_cuda(c.q_nope), K.to_cuda(c.q_pe)
        self.cache, self.table = K.to_cuda(c.kv_cache), K.to_cuda(c.page_table)
        self.lens, self.cu = K.to_cuda(c.seq_lens), K.to_cuda(c.cu)
        self.out = torch.full(self.qn.shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full(self.qn.shape[:2], SENTINEL, dtype=torch.float32, device="cuda")
        dims = mla.make_prefill_dims(self.qn, self.cache, self.table, self.lens)
        self.ws = torch.full((mla.mla_prefill_workspace_size(dims),), 0xFF, dtype=torch.uint8, device="cuda")

    def launch(self, stream=None):
        import paged_mla_decode_09_gb300 as mla

        c = self.c
        mla.mla_prefill(self.qn, self.qp, self.cache, self.table, self.lens, self.cu, c.window, c.sinks, c.scale,
                        c.kv_scale, self.out, self.lse, self.ws, stream)

    def result(self):
        import paged_mla_decode_09_gb300 as mla

        torch.cuda.synchronize()
        status = mla.mla_query_status(self.ws)
        assert not status & (mla.MLA_DEV_TIMEOUT | mla.MLA_DEV_INTERNAL), mla.timeout_diagnostics(self.ws)
        return self.out.float().cpu().numpy().astype(np.float64), self.lse.cpu().numpy().astype(np.float64), status


def check_tokens(c, out, lse, ref=None):
    """Every token of every request against the oracle."""
    ro, rl = ref if ref is not None else oracle.mla_prefill_ref(
        c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, c.window, c.sinks, c.scale, c.kv_scale, c.kv_dtype)
    for b in range(len(c.seq_lens)):
        for i in range(int(c.cu[b + 1] - c.cu[b])):
            t = int(c.cu[b]) + i
            to, tl = K.error_bounds(c, b, i)
            eo, el = np.abs(out[t] - ro[t]), np.abs(lse[t] - rl[t])
            assert np.all(eo <= to), (b, i, float((eo / to).max()), float(eo.max()))
            assert np.all(el <= tl), (b, i, float((el / tl).max()), float(el.max()))
    n = int(c.cu[-1])
    rms = np.sqrt(np.mean(ro[:n] ** 2))
    assert np.sqrt(np.mean((out[:n] - ro[:n]) ** 2)) <= 2.0**-8 * rms  # bounds in the mean: far below the worst case


def run_and_check(c):
    r = Run(c)
    r.launch()
    out, lse, status = r.result()
    assert status == 0
    n = int(c.cu[-1])
    assert np.all(out[n:] == SENTINEL) and np.all(lse[n:] == SENTINEL)  # rows behind the last sequence
    check_tokens(c, out, lse)
    return r


CASES = {
    "one_token": dict(new=[1], total=[1], heads=16),
    "one_head": dict(new=[1], total=[65], heads=1),
    "page_edges": dict(new=[1, 63, 64, 65], total=[64, 63, 128, 129], heads=4),
    "whole_prompts": dict(new=[1, 33, 100], total=[1, 33, 100], heads=16),
    "odd_heads_no_queries": dict(new=[0, 5, 0, 30, 0], total=[70, 200, 1, 500, 0], heads=20),
    "wide_heads": dict(new=[3, 17], total=[130, 1000], heads=128),
    "more_heads_than_rows": dict(new=[2], total=[300], heads=200),
    "pieces": dict(new=[2], total=[20000], heads=16),
    "pieces_of_few": dict(new=[1, 4], total=[9000, 2000], heads=64),
    "many_requests": dict(new=[1 + k % 3 for k in range(150)], total=[40 + 7 * k for k in range(150)], heads=8),
    "full_blocks": dict(new=[70], total=[700], heads=64),
    "full_blocks_pieces": dict(new=[16, 40], total=[6000, 41], heads=32),
    # several blocks per cluster, blocks' last rows in the middle of a warp's
    "many_full_blocks": dict(new=[33] * 8 + [7], total=[90 + 83 * k for k in range(9)], heads=64),
    "many_ragged_blocks": dict(new=[33 + k for k in range(14)], total=[60 + 97 * k for k in range(14)], heads=20),
    "even_blocks": dict(new=[1] * 60, total=[260 + k for k in range(60)], heads=64),  # a cluster each, uncut
    "rows_behind": dict(new=[9, 3], total=[100, 64], heads=16, extra_q=5),
}


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("name", list(CASES))
def test_prefill_parity(name, kv_dtype):
    run_and_check(K.make(seed=len(name), kv_dtype=kv_dtype, **CASES[name]))


WINDOWS = [(1, 0), (1, 3), (33, 4), (64, 64), (100, 70), (129, 0), (500, 1), (2000, 130), (5000, 10000)]


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_prefill_window_parity(window, sinks, kv_dtype):
    run_and_check(K.make([5, 0, 90, 1], [5, 300, 1100, 640], heads=16, window=window, sinks=sinks, kv_dtype=kv_dtype,
                         seed=window + sinks))


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_peaked_scores_rescale_the_output(kv_dtype):
    """Scores ten times as spread: references rise on most pages."""
    run_and_check(K.make([3, 20], [900, 1500], heads=32, kv_dtype=kv_dtype, seed=5, q_gain=10.0))


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("B,H,Q,window,sinks", [(1, 16, 1, 256, 4), (5, 64, 1, 100, 0), (3, 128, 2, 70, 16),
                                                (2, 128, 3, 1, 1), (40, 20, 2, 33, 5)])
def test_decode_window_parity(B, H, Q, window, sinks, kv_dtype):
    import paged_mla_decode_09_gb300 as mla

    total = [Q + (977 * b + 211) % 1500 for b in range(B)]
    c = K.make([Q] * B, total, H, window=window, sinks=sinks, kv_dtype=kv_dtype, seed=B + H)
    r = Run(c)
    qn, qp = r.qn.view(B, Q, H, 512), r.qp.view(B, Q, H, 64)
    ws = torch.full((mla.mla_decode_window_workspace_size(mla.make_dims(qn, r.cache, r.table)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    mla.mla_decode_window(qn, qp, r.cache, r.table, r.lens, window, sinks, c.scale, c.kv_scale,
                          r.out.view(B, Q, H, 512), r.lse.view(B, Q, H), ws)
    torch.cuda.synchronize()
    assert mla.mla_query_status(ws) == 0
    check_tokens(c, r.out.float().cpu().numpy().astype(np.float64), r.lse.cpu().numpy().astype(np.float64))


def test_table_slice_and_repeat_are_bit_identical():
    c = K.make([7, 60, 1], [300, 2000, 5000], heads=32, seed=11)
    r = run_and_check(c)
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


def test_shared_prefix_pages_are_read_in_place():
    """Requests whose tables name the same pages see the same rows."""
    c = K.make([4, 4], [256, 256], heads=16, seed=3)
    c.page_table[1] = c.page_table[0]
    run_and_check(c)


def test_bad_inputs_raise_flags_and_leave_other_requests_alone():
    import paged_mla_decode_09_gb300 as mla

    c = K.make([3, 5, 2], [100, 200, 90], heads=16, seed=9)
    ref = oracle.mla_prefill_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, 0, 0, c.scale)
    r = Run(c)
    r.table[1, 1] = c.kv_cache.shape[0]  # behind the pool
    r.launch()
    out, lse, status = r.result()
    assert status == mla.MLA_DEV_BAD_PAGE_ID
    assert np.allclose(out[[0, 1, 2, 8, 9]], ref[0][[0, 1, 2, 8, 9]], atol=2e-2)

    r = Run(c)
    r.lens[1] = 2  # fewer cached tokens than new ones: three of the five see nothing
    r.launch()
    out, lse, status = r.result()
    assert status == mla.MLA_DEV_BAD_SEQ_LEN
    assert np.all(out[3:6] == 0) and np.all(lse[3:6] == -np.inf) and np.all(np.isfinite(out[6:8]))
    assert np.allclose(out[[0, 1, 2, 8, 9]], ref[0][[0, 1, 2, 8, 9]], atol=2e-2)

    r = Run(c)
    r.lens[2] = 10**6  # beyond the table: clamped to it
    r.launch()
    assert r.result()[2] & mla.MLA_DEV_BAD_SEQ_LEN

    for cu in ([0, 3, 2, 10], [0, 3, 8, 11], [1, 3, 8, 10], [0, -5, 8, 10]):
        r = Run(c)
        r.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        r.launch()
        out, lse, status = r.result()
        assert status & mla.MLA_DEV_BAD_QUERY_RANGE, cu
    # the requests left out were not written
    r = Run(c)
    r.cu.copy_(torch.tensor([0, 3, 8, 11], dtype=torch.int32))
    r.launch()
    out, lse, _ = r.result()
    assert np.all(out[8:] == SENTINEL) and np.allclose(out[:8], ref[0][:8], atol=2e-2)


def test_captured_call_follows_its_inputs():
    """A captured call reads lengths, offsets and tables anew at each replay;
    two graphs that share a workspace run one after the other."""
    a = K.make([6, 2, 9], [500, 64, 1300], heads=16, seed=21)
    b = K.make([1, 15, 1], [33, 1000, 700], heads=16, seed=22)
    width = max(a.page_table.shape[1], b.page_table.shape[1])
    r = Run(a)
    table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    pool = torch.zeros((max(a.kv_cache.shape[0], b.kv_cache.shape[0]), 64, 576), dtype=torch.bfloat16, device="cuda")
    r.table, r.cache = table, pool
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
    for k, c in enumerate((a, b, a)):
        r.table.fill_(-1)
        r.table[:, :c.page_table.shape[1]] = K.to_cuda(c.page_table)
        r.cache[:c.kv_cache.shape[0]] = K.to_cuda(c.kv_cache)
        r.lens.copy_(K.to_cuda(c.seq_lens))
        r.cu.copy_(K.to_cuda(c.cu))
        r.qn.zero_()
        r.qn[:c.q_nope.shape[0]] = K.to_cuda(c.q_nope)[:r.qn.shape[0]]
        r.qp[:c.q_pe.shape[0]] = K.to_cuda(c.q_pe)[:r.qp.shape[0]]
        graphs[k % 2].replay()
        graphs[(k + 1) % 2].replay()
        out, lse, status = r.result()
        assert status == 0
        check_tokens(c, out, lse)


def test_two_streams_with_their_own_workspaces():
    cs = [K.make([50], [1500], heads=16, seed=31), K.make([3, 3], [4000, 200], heads=64, window=300, sinks=2, seed=32)]
    rs = [run_and_check(c) for c in cs]
    want = [(r.out.clone(), r.lse.clone()) for r in rs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for r, s in zip(rs, streams):
            r.launch(stream=s)
    for r, (o, l) in zip(rs, want):
        r.result()
        assert torch.equal(r.out, o) and torch.equal(r.lse, l)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 4)])
def test_many_blocks_per_cluster(window, sinks, kv_dtype):
    """More row blocks than clusters, so that clusters walk from one to the
    next: sampled tokens of chunks of 300 and 129 tokens, 128 heads."""
    c = K.make([300, 129], [3500, 129], 128, window=window, sinks=sinks, kv_dtype=kv_dtype, seed=41)
    r = Run(c)
    r.launch()
    out, lse, status = r.result()
    assert status == 0 and np.all(np.isfinite(out)) and np.all(np.isfinite(lse))
    for b, tokens in ((0, (0, 1, 63, 150, 298, 299)), (1, (0, 5, 64, 128))):
        for i in tokens:
            t = int(c.cu[b]) + i
            keys = oracle.seen_keys(int(c.seq_lens[b] - (c.cu[b + 1] - c.cu[b])) + i, window, sinks)
            rows = oracle.cache_rows_at(c.kv_cache, c.page_table[b], keys, kv_dtype, c.kv_scale)
            q = np.concatenate([oracle.bf16_bits_to_f64(c.q_nope[t]), oracle.bf16_bits_to_f64(c.q_pe[t])], axis=-1)
            ro, rl = oracle.attend(q, rows, rows.shape[0], c.scale)
            to, tl = K.error_bounds(c, b, i)
            assert np.all(np.abs(out[t] - ro) <= to) and np.all(np.abs(lse[t] - rl) <= tl), (b, i)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_pairs_with_garbage_behind_every_sequence_repeat_bit_for_bit(kv_dtype):
    """A pair's two CTAs each clear (bf16) or expand (e4m3) their half of a
    page with ordinary stores, which the other CTA's products read: NaN behind
    each of many sequences must never show, call after call."""
    c = K.make([5] * 24, [5 + (61 * k) % 700 for k in range(24)], 64, kv_dtype=kv_dtype, seed=77)
    r = run_and_check(c)
    out, lse = r.out.clone(), r.lse.clone()
    differs = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(300):
        r.out.zero_()
        r.launch()
        differs |= (r.out != out).any() | (r.lse != lse).any()
    assert r.result()[2] == 0 and not bool(differs)


@pytest.mark.parametrize("heads", [16, 160])
def test_zero_queries_under_a_tiny_cache_scale(heads):
    """An e4m3 cache's queries carry their row's power-of-two scale, 2^-107 for
    a row of zeros; times a small kv_scale that is below what fp32 holds.  The
    row's scores are 0, its weights even, also where a page is only partly seen."""
    c = K.make([3, 1], [200, 70], heads=heads, kv_dtype="fp8_e4m3", window=90, sinks=2, seed=51)
    c.kv_scale = 1e-13
    c.q_nope[:, ::2] = 0
    c.q_pe[:, ::2] = 0
    run_and_check(c)


@pytest.mark.parametrize("spikes", [(0,), (0, 330)])
@pytest.mark.parametrize("gap", [10.0, 17.0, 22.0, 30.0])
@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("B,Q,H", [(90, 1, 64), (40, 3, 128), (1, 2, 64)])
def test_tokens_that_take_the_weight_and_give_nothing(B, Q, H, kv_dtype, gap, spikes):
    """Sink tokens: scores `gap` above the others' (weights e^-gap of theirs for
    the rest, down to 1e-13) and values of 0, so that the outputs are what the
    others give.  A bf16 cache's weights keep their 8 bits however small they
    are.  An e4m3 cache's are f16 against a reference that is no more than the
    row's greatest score, so that rounding moves a weight by at most 2^-11 of
    itself or, below 2^-14, half of f16's least step 2^-24, times the greatest
    weight: 2^-25 w_max |v| more per key."""
    c = K.make([Q] * B, [640] * B, H, kv_dtype=kv_dtype, seed=61, q_gain=0.2)
    one = W.f32_to_bf16_bits(np.array([16.0], dtype=np.float32))[0]
    c.q_pe[:] = 0
    c.q_pe[:, :, 0] = one
    top = np.float32(gap / (16.0 * c.scale))
    zero_code = c.kv_cache.dtype.type(0)
    for b in range(B):
        for p in range(10):
            c.kv_cache[c.page_table[b, p], :, 512:] = zero_code
        for t in spikes:
            row = c.kv_cache[c.page_table[b, t // 64], t % 64]
            row[:] = zero_code
            if kv_dtype == "bf16":
                row[512] = W.f32_to_bf16_bits(np.array([top], dtype=np.float32))[0]
            else:
                row[512] = torch.tensor([top / c.kv_scale]).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).item()
    if kv_dtype != "bf16":  # a scale under which the sinks' keys fit
        c.kv_scale = max(c.kv_scale, float(top) / 448.0 * 1.001)
        for b in range(B):
            for t in spikes:
                c.kv_cache[c.page_table[b, t // 64], t % 64, 512] = \
                    torch.tensor([top / c.kv_scale]).to(torch.float8_e4m3fn).view(torch.uint8).item()
    r = Run(c)
    r.launch()
    out, lse, status = r.result()
    assert status == 0
    for b in sorted({0, B // 2, B - 1}):
        for i in range(Q):
            t = b * Q + i
            keys = oracle.seen_keys(640 - Q + i, 0, 0)
            rows = oracle.cache_rows_at(c.kv_cache, c.page_table[b], keys, kv_dtype, c.kv_scale)
            q = np.concatenate([oracle.bf16_bits_to_f64(c.q_nope[t]), oracle.bf16_bits_to_f64(c.q_pe[t])], axis=-1)
            ro, rl = oracle.attend(q, rows, rows.shape[0], c.scale)
            to, tl = K.error_bounds(c, b, i)
            if kv_dtype != "bf16":
                w_max = np.exp(((q @ rows.T) * c.scale).max(axis=1) - rl)
                to = to + 2.0**-25 * w_max[:, None] * np.abs(rows[:, :512]).sum(axis=0)
            assert np.all(np.abs(lse[t] - rl) <= tl)
            assert np.all(np.abs(out[t] - ro) <= to), (b, i, float((np.abs(out[t] - ro) / to).max()))
