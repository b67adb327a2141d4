"""mla_prefill and mla_decode_window where the schedule takes its large form
(more than 256 requests or row blocks): several rounds of its scans, requests
without queries, and the arrays that then live in global memory (above 2048
requests, above 8192 blocks).  Tokens against the formula in 64 bits on the
device, element by element with the bounds of chunk_cases.error_bounds."""
import numpy as np
import pytest

from chunk_cases import SCALE

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


class Case:
    """new[b] query tokens of total[b] cached ones over a pool of `pool` pages
    that requests share at random; NaN nowhere, extra_q rows behind the last."""

    def __init__(self, new, total, H, window=0, sinks=0, kv_dtype="bf16", pool=400, seed=0, extra_q=3):
        import paged_mla_decode_09_gb300 as mla

        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.new, self.total, self.H, self.window, self.sinks = list(new), list(total), H, window, sinks
        B, self.T = len(new), sum(new)
        width = max(1, -(-max(total) // 64))
        self.table = torch.randint(0, pool, (B, width), generator=gen, device="cuda", dtype=torch.int32)
        for b in range(B):
            self.table[b, -(-total[b] // 64):] = -1
        x = rand(pool, 64, 576).bfloat16()
        self.kv_scale, self.f8 = 1.0, kv_dtype != "bf16"
        if self.f8:
            self.kv_scale = float(x.abs().max()) / 448.0
            x = (x.float() / self.kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.cache = x
        self.qn = torch.empty(self.T + extra_q, H, 512, dtype=torch.bfloat16, device="cuda")
        self.qp = torch.empty(self.T + extra_q, H, 64, dtype=torch.bfloat16, device="cuda")
        for t in range(0, self.T + extra_q, 1024):
            self.qn[t:t + 1024] = rand(*self.qn[t:t + 1024].shape)
            self.qp[t:t + 1024] = rand(*self.qp[t:t + 1024].shape)
        self.lens = torch.tensor(self.total, dtype=torch.int32, device="cuda")
        self.cu_np = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.cu = torch.from_numpy(self.cu_np).cuda()
        self.out = torch.full_like(self.qn, SENTINEL)
        self.lse = torch.full((self.T + extra_q, H), SENTINEL, device="cuda")
        n = mla.mla_prefill_workspace_size(mla.make_prefill_dims(self.qn, self.cache, self.table, self.lens))
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def blocks(self):
        B, rows = len(self.new), self.qn.shape[0] * self.H
        return rows // (256 if rows > 128 * B else 128) + B

    def launch(self):
        import paged_mla_decode_09_gb300 as mla

        mla.mla_prefill(self.qn, self.qp, self.cache, self.table, self.lens, self.cu, self.window, self.sinks, SCALE,
                        self.kv_scale, self.out, self.lse, self.ws)
        return self.status()

    def status(self):
        import paged_mla_decode_09_gb300 as mla

        torch.cuda.synchronize()
        st = mla.mla_query_status(self.ws)
        assert not st & (mla.MLA_DEV_TIMEOUT | mla.MLA_DEV_INTERNAL), mla.timeout_diagnostics(self.ws)
        return st

    def check(self, tokens):
        """Tokens (request, index) against the formula."""
        for b, i in tokens:
            t = int(self.cu_np[b]) + i
            pos = self.total[b] - self.new[b] + i
            k = torch.arange(pos + 1, device="cuda")
            if self.window:
                k = k[(k > pos - self.window) | (k < self.sinks)]
            rows = self.cache[self.table[b, k // 64].long(), k % 64]
            rows = rows.view(torch.float8_e4m3fn).double() * self.kv_scale if self.f8 else rows.double()
            q = torch.cat([self.qn[t], self.qp[t]], dim=-1).double()
            s = q @ rows.T * SCALE
            lse = torch.logsumexp(s, dim=1)
            w = torch.exp(s - lse[:, None])
            out, mean_abs = w @ rows[:, :512], w @ rows[:, :512].abs()
            d = 584 * 2.0**-23 * (q.abs() @ rows.abs().T).amax(dim=1) * SCALE
            if self.f8:
                d = d + 2.0**-17 * q.abs().amax(dim=1) * rows.abs().sum(dim=1).max() * SCALE
            acc = (len(k) / 16 + 64) * 2.0**-23
            out_tol = 2.0**-8 * out.abs() + (2.0**-8 + acc + 2 * d)[:, None] * mean_abs + 1e-30
            lse_tol = d + acc + 8 * 2.0**-23 * (lse.abs() + 1)
            eo, el = (self.out[t].double() - out).abs(), (self.lse[t].double() - lse).abs()
            assert bool((eo <= out_tol).all()), (b, i, float((eo / out_tol).max()))
            assert bool((el <= lse_tol).all()), (b, i, float((el / lse_tol).max()))

    def everything(self):
        return [(b, i) for b in range(len(self.new)) for i in range(self.new[b])]

    def some(self, n, seed=0):
        """A request's first and last tokens, tokens at block borders, and others."""
        rng = np.random.default_rng(seed)
        picks = []
        for b in rng.permutation([b for b in range(len(self.new)) if self.new[b]])[:n]:
            m = self.new[b]
            picks += [(int(b), i) for i in {0, m - 1, min(m - 1, 256 // self.H), int(rng.integers(m)), int(rng.integers(m))}]
        return picks


def ragged(B, most, longest):
    new = [(7 * b) % (most + 1) for b in range(B)]
    return new, [max(1, n) + (131 * b) % longest for b, n in enumerate(new)]


WINDOWS = [(0, 0), (70, 3)]


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("B,most,H,longest", [
    (300, 3, 8, 500),     # two rounds of 1024 threads for the blocks of some, one for the requests
    (257, 2, 4, 200),     # the first batch of the large form
    (1100, 2, 4, 150),    # two rounds for the requests
    (2100, 1, 2, 100),    # first blocks of requests in global memory
])
def test_many_requests(B, most, H, longest, window, sinks, kv_dtype):
    new, total = ragged(B, most, longest)
    c = Case(new, total, H, window, sinks, kv_dtype, seed=B)
    assert B > 256 and 0 in new
    assert c.launch() == 0
    assert bool((c.out[c.T:] == SENTINEL).all()) and bool((c.lse[c.T:] == SENTINEL).all())
    assert bool(torch.isfinite(c.out.float()).all()) and bool(torch.isfinite(c.lse).all())
    c.check(c.everything())


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_just_above_the_small_form(window, sinks, kv_dtype):
    c = Case([255, 256], [900, 256], 128, window, sinks, kv_dtype, seed=5, extra_q=1)
    assert c.blocks() == 258
    assert c.launch() == 0
    assert bool((c.out[c.T:] == SENTINEL).all())
    c.check(c.some(2) + [(0, i) for i in range(0, 255, 17)] + [(1, i) for i in range(0, 256, 17)])


@pytest.mark.parametrize("kv_dtype,window,sinks", [("bf16", 0, 0), ("fp8_e4m3", 0, 0), ("bf16", 300, 70),
                                                   ("fp8_e4m3", 300, 70)])
def test_block_sums_in_global_memory(kv_dtype, window, sinks):
    """Above 8192 blocks of 256 rows: prompts of 5400 to 5700 tokens at once."""
    c = Case([5400, 5563, 5700], [5400, 5600, 5700], 128, window, sinks, kv_dtype, pool=200, seed=6)
    assert c.blocks() > 8192
    assert c.launch() == 0
    assert bool((c.out[c.T:] == SENTINEL).all())
    assert bool(torch.isfinite(c.lse).all())
    c.check(c.some(3) + [(b, i) for b in range(3) for i in range(11, c.new[b], 397)])


def test_requests_and_block_sums_in_global_memory():
    """One token each of 9000 requests, whole outputs."""
    total = [1 + (37 * b) % 300 for b in range(9000)]
    c = Case([1] * 9000, total, 1, kv_dtype="fp8_e4m3", seed=8)
    assert c.blocks() > 8192
    assert c.launch() == 0
    assert bool(torch.isfinite(c.out.float()).all())
    c.check(c.some(2500))


def test_window_decode_of_many_requests():
    import paged_mla_decode_09_gb300 as mla

    B, Q, H = 1300, 2, 16
    total = [Q + (211 * b) % 700 for b in range(B)]
    c = Case([Q] * B, total, H, 100, 5, seed=9, extra_q=0)
    qn, qp = c.qn.view(B, Q, H, 512), c.qp.view(B, Q, H, 64)
    n = mla.mla_decode_window_workspace_size(mla.make_dims(qn, c.cache, c.table))
    c.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    mla.mla_decode_window(qn, qp, c.cache, c.table, c.lens, 100, 5, SCALE, 1.0, c.out.view(B, Q, H, 512),
                          c.lse.view(B, Q, H), c.ws)
    assert c.status() == 0
    c.check(c.some(400))


def test_bad_offsets_among_many_requests():
    import paged_mla_decode_09_gb300 as mla

    new, total = ragged(1100, 2, 150)
    c = Case(new, total, 4, seed=10)
    assert c.launch() == 0
    out, lse = c.out.clone(), c.lse.clone()
    # a decrease or an end behind the queries: the two requests at that offset
    # may lose their rows, all others keep their results
    for value, at in ((-5, 600), (c.T + 9, 601)):
        cu = c.cu_np.copy()
        cu[at] = value
        c.cu.copy_(torch.from_numpy(cu))
        c.out.fill_(SENTINEL)
        assert c.launch() & mla.MLA_DEV_BAD_QUERY_RANGE
        for rows in (slice(0, int(c.cu_np[at - 1])), slice(int(c.cu_np[at + 1]), c.T)):
            assert torch.allclose(c.out[rows].float(), out[rows].float(), atol=2e-2)
            assert torch.allclose(c.lse[rows], lse[rows], atol=1e-2)
    # ranges that overlap everywhere: flagged, and nothing beyond the tensors is written
    cu = np.zeros(1101, dtype=np.int32)
    cu[1::2] = c.T
    c.cu.copy_(torch.from_numpy(cu))
    c.out.fill_(SENTINEL)
    assert c.launch() & mla.MLA_DEV_BAD_QUERY_RANGE
    assert bool((c.out[c.T:] == SENTINEL).all())
