"""GPU tests of mla_attn_mass and mla_evict against the oracle, and a run of
the cache's operators together as a serving loop uses them."""
import numpy as np
import pytest

import chunk_cases as K
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


# ---------------------------------------------------------------- mass

class Mass:
    def __init__(self, c, B, Q, H, lse, cols=None, seed=0):
        import paged_mla_decode_09_gb300 as mla

        self.c, self.B, self.Q, self.H = c, B, Q, H
        cols = cols or c.page_table.shape[1] * 64
        rng = np.random.default_rng(seed)
        self.mass_np = rng.random((B, cols)).astype(np.float32)
        self.lse_np = lse.astype(np.float32)
        self.qn, self.qp = K.to_cuda(c.q_nope).view(B, Q, H, 512), K.to_cuda(c.q_pe).view(B, Q, H, 64)
        self.cache, self.table, self.lens = K.to_cuda(c.kv_cache), K.to_cuda(c.page_table), K.to_cuda(c.seq_lens)
        self.lse, self.mass = K.to_cuda(self.lse_np), K.to_cuda(self.mass_np)
        n = mla.mla_attn_mass_workspace_size(mla.make_dims(self.qn, self.cache, self.table))
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        self.out = torch.full((B, cols), -1.0, device="cuda")

    def launch(self, fresh, mass="in", stream=None):
        import paged_mla_decode_09_gb300 as mla

        mla.mla_attn_mass(self.qn, self.qp, self.cache, self.table, self.lens, self.lse, fresh, self.c.scale,
                          self.c.kv_scale, self.mass if mass == "in" else mass, self.out, self.ws, stream)

    def status(self):
        import paged_mla_decode_09_gb300 as mla

        torch.cuda.synchronize()
        st = mla.mla_query_status(self.ws)
        assert not st & mla.MLA_DEV_TIMEOUT, mla.timeout_diagnostics(self.ws)
        return st


def lse_of(c, B, Q, H):
    _, lse = oracle.mla_prefill_ref(c.q_nope, c.q_pe, c.kv_cache, c.page_table, c.seq_lens, c.cu, 0, 0, c.scale,
                                    c.kv_scale, c.kv_dtype)
    return lse.reshape(B, Q, H)


def check_mass(m, fresh, mass=None):
    """|gpu - exact| per key: every weight e^(s - lse) carries the score's error
    (584 fp32 operations on at most S1 = sum |q||k| scale; an e4m3 cache adds
    2^-17 of the row's largest |q| per value), 8 roundings of exponent and
    result, and the sum of R weights and the key's earlier value R + 1
    roundings."""
    c = m.c
    start = np.zeros_like(m.mass_np) if mass is None else m.mass_np
    ref = oracle.attn_mass_ref(c.q_nope.reshape(m.B, m.Q, m.H, 512), c.q_pe.reshape(m.B, m.Q, m.H, 64), c.kv_cache,
                               c.page_table, c.seq_lens, m.lse_np, fresh, c.scale, c.kv_scale, c.kv_dtype, start)
    got = m.out.cpu().numpy().astype(np.float64)
    for b in range(m.B):
        L = int(c.seq_lens[b])
        rows = oracle.cache_rows_at(c.kv_cache, c.page_table[b], np.arange(L), c.kv_dtype, c.kv_scale)
        q = np.concatenate([oracle.bf16_bits_to_f64(c.q_nope), oracle.bf16_bits_to_f64(c.q_pe)], axis=-1)
        q = q.reshape(m.B, m.Q * m.H, 576)[b]
        d = 584 * 2.0**-23 * (np.abs(q) @ np.abs(rows).T).max() * c.scale
        if c.kv_dtype != "bf16":
            d += 2.0**-17 * np.abs(q).max() * np.abs(rows).sum(axis=1).max() * c.scale
        d += 2.0**-23 * (8 + 4 * np.abs(m.lse_np[b][np.isfinite(m.lse_np[b])]).max(initial=0.0) + m.Q * m.H + 1)
        tol = d * np.abs(ref[b, :L]) + 1e-30
        e = np.abs(got[b, :L] - ref[b, :L])
        assert np.all(e <= tol), (b, float((e / tol).max()))
        assert np.all(got[b, L:] == -1.0)  # entries behind the sequence
    return ref


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("B,Q,H,total", [
    (1, 1, 1, [1]), (1, 1, 16, [700]), (3, 1, 64, [64, 65, 1000]), (2, 1, 128, [129, 63]), (2, 3, 20, [300, 3]),
    (2, 5, 128, [700, 5]), (1, 32, 16, [2500]), (40, 1, 8, [1 + 37 * k for k in range(40)]), (1, 2, 200, [1200]),
    (3, 3, 64, [200, 3, 129]), (2, 64, 3, [64, 257]), (1, 129, 1, [130]),
])
def test_mass_parity(B, Q, H, total, kv_dtype):
    c = K.make([Q] * B, total, H, kv_dtype=kv_dtype, seed=B + Q + H)
    m = Mass(c, B, Q, H, lse_of(c, B, Q, H), seed=1)
    m.launch(Q)
    assert m.status() == 0
    check_mass(m, Q, "in")
    if Q > 1 or H > 1:  # all weights of a row add to one
        m.launch(0, None)
        m.status()
        got = m.out.cpu().numpy()
        for b in range(B):
            assert abs(got[b, :total[b]].sum() - Q * H) <= 1e-3 * Q * H


def test_mass_accumulates_in_place_and_repeats_bit_for_bit():
    c = K.make([2, 2], [900, 130], 64, seed=8)
    m = Mass(c, 2, 2, 64, lse_of(c, 2, 2, 64), cols=1024, seed=2)
    m.launch(0)
    assert m.status() == 0
    first = m.out.clone()
    check_mass(m, 0, "in")
    m.out.copy_(m.mass)
    m.launch(0, m.out)  # mass_out is mass
    m.status()
    for b, L in enumerate((900, 130)):
        assert torch.equal(m.out[b, :L], first[b, :L])
        assert torch.equal(m.out[b, L:], m.mass[b, L:])
    m.out.fill_(-1.0)
    m.launch(2**31 - 1)  # everything fresh: as without a mass
    m.status()
    check_mass(m, 2**31 - 1, None)


def test_mass_empty_rows_and_bad_inputs():
    import paged_mla_decode_09_gb300 as mla

    c = K.make([1, 1, 1], [100, 200, 70], 16, seed=4)
    lse = lse_of(c, 3, 1, 16)
    lse[0, 0, 3] = -np.inf  # a row that saw nothing adds nothing
    m = Mass(c, 3, 1, 16, lse, seed=3)
    m.launch(1)
    assert m.status() == 0
    check_mass(m, 1, "in")
    m.table[1, 0] = -7
    m.launch(1)
    assert m.status() == mla.MLA_DEV_BAD_PAGE_ID
    m.table.copy_(K.to_cuda(c.page_table))
    for bad in (0, -5, 10**6):
        m.lens[1] = bad
        m.out.fill_(-1.0)
        m.launch(1)
        assert m.status() & mla.MLA_DEV_BAD_SEQ_LEN
        if bad < 1:
            assert torch.all(m.out[1] == -1.0)
    m.lens.copy_(K.to_cuda(c.seq_lens))
    narrow = Mass(c, 3, 1, 16, lse, cols=100, seed=3)  # 200 tokens, room for 100
    narrow.launch(1)
    assert narrow.status() & mla.MLA_DEV_BAD_SEQ_LEN


# ---------------------------------------------------------------- evict

def evict_case(total, budget, sinks, recent, kv_dtype="bf16", seed=0, positions=True, ties=0.2, width=None):
    rng = np.random.default_rng(seed)
    B = len(total)
    npg = [-(-n // 64) for n in total]
    width = width or max(1, max(npg))
    pages = sum(npg) + 2
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :npg[b]] = ids[at:at + npg[b]]
        at += npg[b]
    if kv_dtype == "bf16":
        cache = rng.integers(0, 1 << 16, size=(pages, 64, 576)).astype(np.uint16)
    else:
        cache = rng.integers(0, 256, size=(pages, 64, 576)).astype(np.uint8)
    cols = width * 64
    mass = np.exp(2 * rng.standard_normal((B, cols))).astype(np.float32)
    mass[rng.random((B, cols)) < ties] = 0.0
    mass[rng.random((B, cols)) < ties] = 0.25
    pos = None
    if positions:
        pos = np.stack([rng.permutation(3 * cols)[:cols] for _ in range(B)]).astype(np.int32)
        pos.sort(axis=1)
        for b in range(B):
            n = total[b]
            mid = pos[b, min(sinks, n):max(min(sinks, n), n - recent)]
            rng.shuffle(mid)
    return dict(mass=mass, positions=pos, seq_lens=np.array(total, dtype=np.int32), page_table=table, kv_cache=cache,
                budget=budget, sinks=sinks, recent=recent, kv_dtype=kv_dtype)


class Evict:
    def __init__(self, e):
        import paged_mla_decode_09_gb300 as mla

        self.e = e
        B, cols = e["mass"].shape
        self.mass, self.lens, self.table = K.to_cuda(e["mass"]), K.to_cuda(e["seq_lens"]), K.to_cuda(e["page_table"])
        self.pos = None if e["positions"] is None else K.to_cuda(e["positions"])
        self.cache = K.to_cuda(e["kv_cache"])
        self.new_lens = torch.full((B,), -9, dtype=torch.int32, device="cuda")
        self.kept = torch.full((B, e["budget"]), -9, dtype=torch.int32, device="cuda")
        self.mass_out = torch.full((B, cols), -2.0, device="cuda")
        self.pos_out = None if self.pos is None else torch.full((B, cols), -9, dtype=torch.int32, device="cuda")
        self.ws = torch.full((mla.mla_evict_workspace_size(B, e["budget"]),), 0xFF, dtype=torch.uint8, device="cuda")

    def launch(self, stream=None):
        import paged_mla_decode_09_gb300 as mla

        e = self.e
        mla.mla_evict(self.mass, self.pos, self.lens, self.table, self.cache, e["budget"], e["sinks"], e["recent"],
                      self.new_lens, self.kept, self.mass_out, self.pos_out, self.ws, stream)

    def status(self):
        import paged_mla_decode_09_gb300 as mla

        torch.cuda.synchronize()
        return mla.mla_query_status(self.ws)

    def bits(self):
        return self.cache.view(torch.int16).cpu().numpy().view(np.uint16) if self.cache.dtype == torch.bfloat16 \
            else self.cache.cpu().numpy()


def check_evict(r):
    e = r.e
    n, kept, mo, po, cache = oracle.evict_ref(e["mass"], e["positions"], e["seq_lens"], e["page_table"], e["kv_cache"],
                                              e["budget"], e["sinks"], e["recent"])
    assert np.array_equal(r.new_lens.cpu().numpy(), n)
    assert np.array_equal(r.kept.cpu().numpy(), kept)
    assert np.array_equal(r.bits(), cache)  # every byte of the pool
    got = r.mass_out.cpu().numpy()
    for b in range(len(n)):
        assert np.array_equal(got[b, :n[b]], mo[b, :n[b]], equal_nan=True) and np.all(got[b, n[b]:] == -2.0)
        if r.pos_out is not None:
            gp = r.pos_out.cpu().numpy()
            assert np.array_equal(gp[b, :n[b]], po[b, :n[b]]) and np.all(gp[b, n[b]:] == -9)


EVICT = [
    dict(total=[1], budget=1, sinks=0, recent=0),
    dict(total=[2], budget=1, sinks=0, recent=1),
    dict(total=[600], budget=512, sinks=4, recent=128),
    dict(total=[65, 64, 0, 63, 200], budget=64, sinks=1, recent=10),
    dict(total=[700, 100, 1500], budget=129, sinks=0, recent=0),
    dict(total=[700, 100, 1500], budget=129, sinks=129, recent=0),
    dict(total=[700, 100, 1500], budget=129, sinks=0, recent=129),
    dict(total=[5000, 1025, 1024, 1023], budget=1000, sinks=16, recent=500),
    dict(total=[3000], budget=2999, sinks=2, recent=7),
    dict(total=[300 + k for k in range(50)], budget=280, sinks=4, recent=30),
    dict(total=[9000, 8191], budget=4000, sinks=4, recent=300),           # eight blocks a request
    dict(total=[2100, 4100, 50, 3000, 1] * 8, budget=2000, sinks=1, recent=9),  # two
]


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict_exact(case, kv_dtype):
    for positions in (True, False):
        r = Evict(evict_case(**EVICT[case], kv_dtype=kv_dtype, seed=case, positions=positions))
        r.launch()
        assert r.status() == 0
        check_evict(r)


def test_evict_all_equal_and_special_weights():
    e = evict_case([400, 300], 150, 0, 0, seed=1, positions=False)
    e["mass"][0] = 0.0                      # ties: the first 150 slots stay
    e["mass"][0, ::3] = -0.0
    e["mass"][1] = np.nan                   # NaN last, ties by slot
    e["mass"][1, 200:290] = 1.0
    e["mass"][1, 7] = np.inf
    e["mass"][1, 299] = -np.inf
    r = Evict(e)
    r.launch()
    assert r.status() == 0
    check_evict(r)
    assert r.kept[0].cpu().tolist() == list(range(150))


@pytest.mark.parametrize("positions", [True, False])
def test_evict_longer_than_shared_memory(positions):
    """More tokens than a cluster of eight blocks keeps keys of (8 x 20K)."""
    r = Evict(evict_case([170000], 3000, 4, 100, kv_dtype="fp8_e4m3", seed=2, positions=positions))
    r.launch()
    assert r.status() == 0
    check_evict(r)


def test_evict_longer_than_shared_memory_in_place():
    e = evict_case([170000, 90], 3000, 4, 100, kv_dtype="fp8_e4m3", seed=3)
    r = Evict(e)
    r.mass_out, r.pos_out, r.new_lens = r.mass, r.pos, r.lens
    r.launch()
    assert r.status() == 0
    n, kept, mo, po, cache = oracle.evict_ref(e["mass"], e["positions"], e["seq_lens"], e["page_table"], e["kv_cache"],
                                              3000, 4, 100)
    assert np.array_equal(r.lens.cpu().numpy(), n) and np.array_equal(r.kept.cpu().numpy(), kept)
    assert np.array_equal(r.mass.cpu().numpy(), mo) and np.array_equal(r.pos.cpu().numpy(), po)
    assert np.array_equal(r.bits(), cache)


def test_evict_in_place_outputs():
    e = evict_case([700, 64, 1300], 200, 4, 40, seed=6)
    r = Evict(e)
    r.mass_out, r.pos_out, r.new_lens = r.mass, r.pos, r.lens
    r.launch()
    assert r.status() == 0
    n, kept, mo, po, cache = oracle.evict_ref(e["mass"], e["positions"], e["seq_lens"], e["page_table"], e["kv_cache"],
                                              200, 4, 40)
    assert np.array_equal(r.lens.cpu().numpy(), n) and np.array_equal(r.kept.cpu().numpy(), kept)
    assert np.array_equal(r.mass.cpu().numpy(), mo) and np.array_equal(r.pos.cpu().numpy(), po)
    assert np.array_equal(r.bits(), cache)


def test_evict_flags_bad_lengths_and_pages():
    import paged_mla_decode_09_gb300 as mla

    e = evict_case([700, 300], 200, 0, 0, seed=7, positions=False)
    r = Evict(e)
    r.lens[1] = -3
    r.launch()
    assert r.status() == mla.MLA_DEV_BAD_SEQ_LEN
    assert r.new_lens.cpu().tolist() == [200, 0]
    r = Evict(e)
    r.lens[0] = 10**7
    r.launch()  # clamped to what the table and the rows hold
    assert r.status() == mla.MLA_DEV_BAD_SEQ_LEN and r.new_lens.cpu().tolist() == [200, 200]
    r = Evict(e)
    r.table[0, 8] = e["kv_cache"].shape[0]
    r.launch()
    assert r.status() == mla.MLA_DEV_BAD_PAGE_ID
    r = Evict(e)
    r.table[1, 0] = -1
    r.launch()
    assert r.status() == mla.MLA_DEV_BAD_PAGE_ID


# ------------------------------------------------- the operators together

@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_serving_loop(kv_dtype):
    """Cache write, prompt chunk, mass, eviction, then decode steps (one of
    them over a window) on the shortened cache, captured into one graph and
    replayed: every step against the oracle on the oracle's own state."""
    import paged_mla_decode_09_gb300 as mla
    from paged_mla_decode_09_gb300 import workloads as W

    rng = np.random.default_rng(12)
    B, H, new, budget, sinks, recent, cols = 3, 16, [150, 40, 260], 130, 2, 20, 320
    width = cols // 64
    pages = B * width
    table_np = rng.permutation(pages).astype(np.int32).reshape(B, width)
    f8 = kv_dtype != "bf16"
    cache_np = np.zeros((pages, 64, 576), dtype=np.uint8 if f8 else np.uint16)
    kv_scale = 0.02 if f8 else 1.0
    scale = K.SCALE
    bits = lambda *shape: W.f32_to_bf16_bits(rng.standard_normal(shape, dtype=np.float32))  # noqa: E731
    cache, table = K.to_cuda(cache_np), K.to_cuda(table_np)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens_np = np.array(new, dtype=np.int32)
    lens = K.to_cuda(lens_np)

    # prompts: the cache write takes one count per call, so it runs request by request
    for b in range(B):
        rows = bits(1, new[b], 576)
        mla.mla_kv_pack(K.to_cuda(rows), table[b:b + 1], lens[b:b + 1], kv_scale, cache, status)
        cache_np, st = oracle.kv_pack_ref(rows, table_np[b:b + 1], lens_np[b:b + 1], kv_scale, cache_np, kv_dtype)
        assert st == 0
    T = sum(new)
    qn, qp = bits(T, H, 512), bits(T, H, 64)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    c = K.Chunk(qn, qp, cache_np, table_np, lens_np, cu, 0, 0, kv_dtype, kv_scale, scale)
    out = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, H, device="cuda")
    q_d, p_d, cu_d = K.to_cuda(qn), K.to_cuda(qp), K.to_cuda(cu)
    ws = torch.empty(mla.mla_prefill_workspace_size(mla.make_prefill_dims(q_d, cache, table, lens)), dtype=torch.uint8,
                     device="cuda")
    mla.mla_prefill(q_d, p_d, cache, table, lens, cu_d, 0, 0, scale, kv_scale, out, lse, ws)
    torch.cuda.synchronize()
    assert mla.mla_query_status(ws) == 0 and status.item() == 0
    ro, rl = oracle.mla_prefill_ref(qn, qp, cache_np, table_np, lens_np, cu, 0, 0, scale, kv_scale, kv_dtype)
    for b in range(B):
        for i in (0, new[b] - 1):
            t = cu[b] + i
            to, tl = K.error_bounds(c, b, i)
            assert np.all(np.abs(out[t].double().cpu().numpy() - ro[t]) <= to)
            assert np.all(np.abs(lse[t].double().cpu().numpy() - rl[t]) <= tl)

    # mass of the prompts' last 8 tokens, then the eviction
    last = np.concatenate([np.arange(cu[b + 1] - 8, cu[b + 1]) for b in range(B)])
    q8, p8 = qn[last].reshape(B, 8, H, 512), qp[last].reshape(B, 8, H, 64)
    lse8 = lse[torch.from_numpy(last).cuda()].view(B, 8, H).contiguous()
    mass = torch.zeros(B, cols, device="cuda")
    pos = torch.arange(cols, dtype=torch.int32, device="cuda").repeat(B, 1)
    kept = torch.empty(B, budget, dtype=torch.int32, device="cuda")
    wsm = torch.empty(256, dtype=torch.uint8, device="cuda")
    wse = torch.empty(mla.mla_evict_workspace_size(B, budget), dtype=torch.uint8, device="cuda")
    mla.mla_attn_mass(K.to_cuda(q8), K.to_cuda(p8), cache, table, lens, lse8, 0, scale, kv_scale, None, mass, wsm)
    mass_np, pos_np = mass.cpu().numpy(), pos.cpu().numpy()
    ref_mass = oracle.attn_mass_ref(q8, p8, cache_np, table_np, lens_np, lse8.cpu().numpy(), 0, scale, kv_scale,
                                    kv_dtype, np.zeros((B, cols)))
    assert np.allclose(mass_np, ref_mass, rtol=1e-3, atol=1e-6)
    mla.mla_evict(mass, pos, lens, table, cache, budget, sinks, recent, lens, kept, mass, pos, wse)

    def evict_oracle():
        nonlocal lens_np, mass_np, pos_np, cache_np
        n, k, mass_np, pos_np, cache_np = oracle.evict_ref(mass_np, pos_np, lens_np, table_np, cache_np, budget, sinks,
                                                           recent)
        lens_np = n
        assert np.array_equal(lens.cpu().numpy(), n) and np.array_equal(kept.cpu().numpy(), k)
        got = cache.view(torch.int16).cpu().numpy().view(np.uint16) if not f8 else cache.cpu().numpy()
        assert np.array_equal(got, cache_np)
        assert mla.mla_query_status(wse) == 0

    torch.cuda.synchronize()
    evict_oracle()

    # one decode step, captured: lengths + 1, cache write, attention, mass, eviction
    rows_d = torch.empty(B, 1, 576, dtype=torch.bfloat16, device="cuda")
    q1, p1 = torch.empty(B, 1, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(
        B, 1, H, 64, dtype=torch.bfloat16, device="cuda")
    o1, l1 = torch.empty_like(q1), torch.empty(B, 1, H, device="cuda")
    next_pos = torch.tensor(new, dtype=torch.int32, device="cuda")
    dims = mla.make_dims(q1, cache, table)
    wsd = torch.empty(mla.mla_decode_workspace_size(dims), dtype=torch.uint8, device="cuda")
    wsw = torch.empty(mla.mla_decode_window_workspace_size(dims), dtype=torch.uint8, device="cuda")
    ow, lw = torch.empty_like(q1), torch.empty_like(l1)
    window = 33

    def step():
        pos.scatter_(1, lens.long()[:, None], next_pos[:, None])
        next_pos.add_(1)
        lens.add_(1)
        mla.mla_kv_pack(rows_d, table, lens, kv_scale, cache, status)
        mla.mla_decode(q1, p1, cache, table, lens, 1, scale, kv_scale, o1, l1, wsd)
        mla.mla_decode_window(q1, p1, cache, table, lens, window, sinks, scale, kv_scale, ow, lw, wsw)
        mla.mla_attn_mass(q1, p1, cache, table, lens, l1, 1, scale, kv_scale, mass, mass, wsm)
        mass_before.copy_(mass)
        lens_before.copy_(lens)
        mla.mla_evict(mass, pos, lens, table, cache, budget, sinks, recent, lens, kept, mass, pos, wse)

    mass_before, lens_before = torch.empty_like(mass), torch.empty_like(lens)
    state = [t.clone() for t in (pos, next_pos, lens, cache, mass, kept)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rows_d.zero_(), q1.zero_(), p1.zero_()
    with torch.cuda.stream(side):
        step()  # warm-up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((pos, next_pos, lens, cache, mass, kept), state):
        t.copy_(s)
    torch.cuda.synchronize()
    for k in range(4):
        rows, qn1, qp1 = bits(B, 1, 576), bits(B, 1, H, 512), bits(B, 1, H, 64)
        rows_d.copy_(K.to_cuda(rows)), q1.copy_(K.to_cuda(qn1)), p1.copy_(K.to_cuda(qp1))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            pos_np[b, lens_np[b]] = new[b] + k
        lens_np = (lens_np + 1).astype(np.int32)
        cache_np, st = oracle.kv_pack_ref(rows, table_np, lens_np, kv_scale, cache_np, kv_dtype)
        assert st == 0 and np.array_equal(lens_before.cpu().numpy(), lens_np)
        cu1 = np.arange(B + 1, dtype=np.int32)
        for win, o, l in ((0, o1, l1), (window, ow, lw)):
            cw = K.Chunk(qn1[:, 0], qp1[:, 0], cache_np, table_np, lens_np, cu1, win, sinks, kv_dtype, kv_scale, scale)
            ro, rl = oracle.mla_prefill_ref(cw.q_nope, cw.q_pe, cache_np, table_np, lens_np, cu1, win, sinks, scale,
                                            kv_scale, kv_dtype)
            for b in range(B):
                to, tl = K.error_bounds(cw, b, 0)
                if win:
                    assert np.all(np.abs(o[b, 0].double().cpu().numpy() - ro[b]) <= to)
                    assert np.all(np.abs(l[b, 0].double().cpu().numpy() - rl[b]) <= tl)
                else:  # mla_decode has its own, wider bound
                    tol = 4e-2 if f8 else 1e-2
                    assert np.all(np.abs(o[b, 0].double().cpu().numpy() - ro[b]) <= tol + tol * np.abs(ro[b]))
        mass_now = mass_before.cpu().numpy()
        ref = oracle.attn_mass_ref(qn1, qp1, cache_np, table_np, lens_np, l1.cpu().numpy(), 1, scale, kv_scale, kv_dtype,
                                   mass_np)
        for b in range(B):
            assert np.allclose(mass_now[b, :lens_np[b]], ref[b, :lens_np[b]], rtol=1e-3, atol=1e-6)
        mass_np = mass_now  # the selection is exact on the device's own weights
        evict_oracle()
        assert np.array_equal(pos.cpu().numpy(), pos_np)
    assert status.item() == 0
