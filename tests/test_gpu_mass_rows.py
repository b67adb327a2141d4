"""mla_attn_mass above 128 query rows per request (the keys stay, the rows
stream), against sums of exp(s - lse) in 64 bits: calls whose CTAs walk from
one key tile and request to the next, drafts with few row tiles, and loops of
calls that must agree bit for bit."""
import pytest

from chunk_cases import SCALE

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


class Call:
    """Inputs made on the device; lse is the exact one, rounded to 32 bits."""

    def __init__(self, B, Q, H, lens, kv_dtype, seed):
        import paged_mla_decode_09_gb300 as mla

        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.B, self.Q, self.H, self.lens_py = B, Q, H, list(lens)
        pages = [-(-n // 64) for n in lens]
        width = max(pages)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        ids = torch.randperm(sum(pages), generator=gen, device="cuda").to(torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = ids[at:at + n]
            at += n
        x = torch.cat([rand(min(1024, at - k), 64, 576).bfloat16() for k in range(0, at, 1024)])
        self.kv_scale = 1.0
        self.f8 = kv_dtype != "bf16"
        if self.f8:
            self.kv_scale = float(x.abs().max()) / 448.0
            x = (x.float() / self.kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.cache = x
        self.qn, self.qp = rand(B, Q, H, 512).bfloat16(), rand(B, Q, H, 64).bfloat16()
        self.lens = torch.tensor(self.lens_py, dtype=torch.int32, device="cuda")
        self.mass = torch.rand((B, width * 64), generator=gen, device="cuda")
        self.out = torch.full_like(self.mass, -1.0)
        self.lse = torch.empty(B, Q, H, device="cuda")
        for b in range(B):
            self.lse[b] = torch.logsumexp(self.scores(b)[0], dim=1).view(Q, H).float()
        n = mla.mla_attn_mass_workspace_size(mla.make_dims(self.qn, self.cache, self.table))
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def scores(self, b):
        """Request b's masked scores [Q H, L] in 64 bits, its query rows and its keys."""
        L = self.lens_py[b]
        rows = self.cache[self.table[b, :-(-L // 64)].long()].view(-1, 576)[:L]
        rows = rows.view(torch.float8_e4m3fn).double() * self.kv_scale if self.f8 else rows.double()
        q = torch.cat([self.qn[b], self.qp[b]], dim=-1).view(-1, 576).double()
        s = q @ rows.T * SCALE
        pos = L - self.Q + torch.arange(self.Q, device="cuda").repeat_interleave(self.H)
        s[torch.arange(L, device="cuda")[None] > pos[:, None]] = -torch.inf
        return s, q, rows

    def launch(self, fresh, mass, out):
        import paged_mla_decode_09_gb300 as mla

        mla.mla_attn_mass(self.qn, self.qp, self.cache, self.table, self.lens, self.lse, fresh, SCALE, self.kv_scale,
                          mass, out, self.ws)

    def status(self):
        import paged_mla_decode_09_gb300 as mla

        torch.cuda.synchronize()
        st = mla.mla_query_status(self.ws)
        assert not st & mla.MLA_DEV_TIMEOUT, mla.timeout_diagnostics(self.ws)
        return st

    def check(self, got, fresh, mass):
        """Every weight e^(s - lse) carries the score's error (584 fp32
        operations on at most S1 = sum |q||k| scale), 8 roundings of exponent
        and result with the exponent's own size, and the sum of R weights and
        the earlier value R + 1 roundings (as in the smaller cases' test)."""
        for b, L in enumerate(self.lens_py):
            s, q, rows = self.scores(b)
            want = torch.exp(s - self.lse[b].view(-1, 1).double()).sum(dim=0)
            if mass is not None:
                old = max(0, L - fresh)
                want[:old] += mass[b, :old].double()
            d = 584 * 2.0**-23 * float((q.abs() @ rows.abs().T).max()) * SCALE
            d += 2.0**-23 * (8 + 4 * float(self.lse[b].abs().max()) + self.Q * self.H + 1)
            err = (got[b, :L].double() - want).abs()
            assert bool((err <= d * want + 1e-30).all()), (b, float((err / (d * want)).max()))
            assert bool((got[b, L:] == (-1.0 if mass is not got else mass[b, L:])).all())


BATCHES = [
    (40, 3, 64, [3 + 17 * k for k in range(40)]),                # 200 key tiles, from one request to the next
    (1, 3, 64, [25000]),                                         # two key tiles and more per CTA of one request
    (1, 43, 3, [9000]),                                          # 129 rows
    (70, 2, 128, [2 + (311 * k) % 900 for k in range(70)]),      # 4 row tiles
    (9, 5, 64, [1000 + 400 * k for k in range(9)]),              # 5
    (3, 7, 20, [9001, 64, 7000]),                                # 3, the last of 12 rows
]


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("case", range(len(BATCHES)))
def test_many_key_tiles(case, kv_dtype):
    B, Q, H, lens = BATCHES[case]
    assert sum(-(-n // 128) for n in lens) > 64  # no clusters that share a key tile
    c = Call(B, Q, H, lens, kv_dtype, seed=case)
    fresh = Q // 2
    c.launch(fresh, c.mass, c.out)
    assert c.status() == 0
    c.check(c.out, fresh, c.mass)
    # in place: the same values, entries behind the lengths untouched
    inplace = c.mass.clone()
    c.launch(fresh, inplace, inplace)
    assert c.status() == 0
    for b, L in enumerate(lens):
        assert torch.equal(inplace[b, :L], c.out[b, :L]) and torch.equal(inplace[b, L:], c.mass[b, L:])
    # without an earlier mass
    c.out.fill_(-1.0)
    c.launch(0, None, c.out)
    assert c.status() == 0
    c.check(c.out, 0, None)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("B,Q,H", [(32, 5, 64), (64, 2, 128), (33, 3, 64)])
def test_loops_of_calls_agree_bit_for_bit(B, Q, H, kv_dtype):
    """Few row tiles per key tile over many requests, whose rows come now from
    L2, now from memory: 300 calls, every one as the first."""
    lens = [4000 + (7919 * k) % 8000 for k in range(B)]
    c = Call(B, Q, H, lens, kv_dtype, seed=B)
    c.launch(Q, c.mass, c.out)
    assert c.status() == 0
    c.check(c.out, Q, c.mass)
    first, differs = c.out.clone(), torch.zeros((), dtype=torch.bool, device="cuda")
    flush = torch.empty(1 << 26, dtype=torch.float32, device="cuda")
    for k in range(300):
        if k % 3 == 0:
            flush.zero_()  # beyond L2: the rows come from memory again
        c.out.fill_(-1.0)
        c.launch(Q, c.mass, c.out)
        differs |= (c.out != first).any()
        if k % 50 == 49:
            assert c.status() == 0
    assert not bool(differs)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("B,Q,H,lens", [(2, 8, 64, [1000, 65]), (1, 32, 32, [2048]), (5, 3, 100, [700, 128, 1, 640, 333])])
def test_clusters_that_share_a_key_tile(B, Q, H, lens, kv_dtype):
    """8 and 2 CTAs of a cluster share a key tile; calls one behind the other,
    so that a cluster begins while the kernel before it ends."""
    assert sum(-(-max(lens) // 128) for _ in lens) <= 32
    lens = [max(n, Q) for n in lens]
    c = Call(B, Q, H, lens, kv_dtype, seed=Q)
    c.launch(1, c.mass, c.out)
    assert c.status() == 0
    c.check(c.out, 1, c.mass)
    first, other = c.out.clone(), [torch.full_like(c.out, -1.0) for _ in range(20)]
    for _ in range(10):
        for o in other:
            c.launch(1, c.mass, o)
        assert c.status() == 0
        assert all(torch.equal(o, first) for o in other)
