"""mla_prefill, mla_decode_window, mla_attn_mass and mla_evict at the ends of
what their headers allow: offsets beyond 32 bits in the cache, the queries and
the outputs, calls without any query, a row of NaN, many requests, table
slices, calls at once on two streams, graphs that share a workspace, and a
process whose first call is captured."""
import os
import subprocess
import sys

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


def randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def status(ws):
    import paged_mla_decode_09_gb300 as mla

    torch.cuda.synchronize()
    st = mla.mla_query_status(ws)
    assert not st & (mla.MLA_DEV_TIMEOUT | mla.MLA_DEV_INTERNAL), mla.timeout_diagnostics(ws)
    return st


def check_row(qn, qp, rows, out, lse, f8=False):
    """One token's heads [H, ...] over its seen keys, with the bounds of chunk_cases.error_bounds."""
    q = torch.cat([qn, qp], dim=-1).double()
    s = q @ rows.T * SCALE
    want_lse = torch.logsumexp(s, dim=1)
    w = torch.exp(s - want_lse[:, None])
    want, mean_abs = w @ rows[:, :512], w @ rows[:, :512].abs()
    d = 584 * 2.0**-23 * (q.abs() @ rows.abs().T).amax(dim=1) * SCALE
    if f8:
        d = d + 2.0**-17 * q.abs().amax(dim=1) * rows.abs().sum(dim=1).max() * SCALE
    acc = (rows.shape[0] / 16 + 64) * 2.0**-23
    tol = 2.0**-8 * want.abs() + (2.0**-8 + acc + 2 * d)[:, None] * mean_abs + 1e-30
    assert bool(((out.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - want_lse).abs() <= d + acc + 8 * 2.0**-23 * (want_lse.abs() + 1)).all())


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_cache_offsets_beyond_32_bits(kv_dtype):
    """A pool of more than 2^32 bytes (e4m3) or elements (bf16), the requests'
    pages at its far end: chunk, window, mass and eviction."""
    import paged_mla_decode_09_gb300 as mla

    gen = generator(1)
    f8 = kv_dtype != "bf16"
    pages = 120000
    assert pages * 64 * 576 > 2**32
    cache = torch.empty(pages, 64, 576, dtype=torch.uint8 if f8 else torch.bfloat16, device="cuda")
    lens_py, Q, H = [700, 390], 3, 64
    table = torch.full((2, 11), -1, dtype=torch.int32, device="cuda")
    table[0, :11] = torch.arange(pages - 11, pages, device="cuda").flip(0)
    table[1, :7] = torch.arange(pages - 18, pages - 11, device="cuda")
    x = randn(gen, 18, 64, 576)
    kv_scale = float(x.abs().max()) / 448.0 if f8 else 1.0
    cache[pages - 18:] = (x.float() / kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if f8 else x
    values = (lambda c: c.view(torch.float8_e4m3fn).double() * kv_scale) if f8 else (lambda c: c.double())
    lens = torch.tensor(lens_py, dtype=torch.int32, device="cuda")
    qn, qp = randn(gen, 2, Q, H, 512), randn(gen, 2, Q, H, 64)
    out, lse = torch.zeros_like(qn), torch.zeros(2, Q, H, device="cuda")
    rows = [values(cache[table[b, :-(-n // 64)].long()].view(-1, 576)[:n]) for b, n in enumerate(lens_py)]

    flat = (qn.view(2 * Q, H, 512), qp.view(2 * Q, H, 64), out.view(2 * Q, H, 512), lse.view(2 * Q, H))
    ws = torch.zeros(mla.mla_prefill_workspace_size(mla.make_prefill_dims(flat[0], cache, table, lens)),
                     dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, Q, 2 * Q], dtype=torch.int32, device="cuda")
    wws = torch.zeros(mla.mla_decode_window_workspace_size(mla.make_dims(qn, cache, table)), dtype=torch.uint8,
                      device="cuda")
    mla.mla_decode_window(qn, qp, cache, table, lens, 130, 2, SCALE, kv_scale, out, lse, wws)
    assert status(wws) == 0
    for b, n in enumerate(lens_py):
        for i in range(Q):
            pos = n - Q + i
            t = torch.arange(pos + 1, device="cuda")
            check_row(qn[b, i], qp[b, i], rows[b][t[(t > pos - 130) | (t < 2)]], out[b, i], lse[b, i], f8)
    mla.mla_prefill(flat[0], flat[1], cache, table, lens, cu, 0, 0, SCALE, kv_scale, flat[2], flat[3], ws)
    assert status(ws) == 0
    for b, n in enumerate(lens_py):
        for i in range(Q):
            check_row(qn[b, i], qp[b, i], rows[b][:n - Q + i + 1], out[b, i], lse[b, i], f8)

    mass = torch.zeros(2, 704, device="cuda")
    mws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for heads in (H, 32):  # more than 128 rows, fewer
        sel = [a[:, :, :heads].contiguous() for a in (qn, qp, lse)]
        mla.mla_attn_mass(sel[0], sel[1], cache, table, lens, sel[2], 0, SCALE, kv_scale, None, mass, mws)
        assert status(mws) == 0
        for b, n in enumerate(lens_py):
            assert abs(float(mass[b, :n].double().sum()) - Q * heads) < 1e-3 * Q * heads
            q = torch.cat([sel[0][b], sel[1][b]], dim=-1).view(-1, 576).double()
            s = q @ rows[b].T * SCALE
            pos = n - Q + torch.arange(Q, device="cuda").repeat_interleave(heads)
            s[torch.arange(n, device="cuda")[None] > pos[:, None]] = -torch.inf
            want = torch.exp(s - sel[2][b].view(-1, 1).double()).sum(dim=0)
            assert torch.allclose(mass[b, :n].double(), want, rtol=1e-3, atol=1e-7)

    kept = torch.zeros(2, 256, dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    ews = torch.zeros(mla.mla_evict_workspace_size(2, 256), dtype=torch.uint8, device="cuda")
    mo = torch.zeros_like(mass)
    mla.mla_evict(mass, None, lens, table, cache, 256, 4, 16, new, kept, mo, None, ews)
    assert status(ews) == 0 and new.tolist() == [256, 256]
    for b in range(2):
        moved = values(cache[table[b, :4].long()].view(-1, 576)[:256])
        assert torch.equal(moved, rows[b][kept[b].long()])


def test_queries_and_outputs_beyond_32_bits():
    """33000 tokens of 128 heads over a window: more than 2^31 query and
    output values."""
    import paged_mla_decode_09_gb300 as mla

    gen = generator(2)
    T, H, window, sinks = 33000, 128, 64, 3
    assert T * H * 512 > 2**31
    width = -(-T // 64)
    cache = torch.cat([randn(gen, n, 64, 576) for n in (256, width - 256)])
    table = torch.randperm(width, generator=gen, device="cuda").to(torch.int32)[None]
    qn = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda")
    qp = torch.empty(T, H, 64, dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 2000):
        qn[t:t + 2000] = randn(gen, *qn[t:t + 2000].shape)
        qp[t:t + 2000] = randn(gen, *qp[t:t + 2000].shape)
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(qn), torch.zeros(T, H, device="cuda")
    ws = torch.zeros(mla.mla_prefill_workspace_size(mla.make_prefill_dims(qn, cache, table, lens)), dtype=torch.uint8,
                     device="cuda")
    mla.mla_prefill(qn, qp, cache, table, lens, cu, window, sinks, SCALE, 1.0, out, lse, ws)
    assert status(ws) == 0
    for i in (0, 1, 66, 16383, 16384, 32767, 32768, T - 1):
        t = torch.arange(i + 1, device="cuda")
        t = t[(t > i - window) | (t < sinks)]
        check_row(qn[i], qp[i], cache[table[0, t // 64].long(), t % 64].double(), out[i], lse[i])

    # the mass of all those rows, most of which saw nothing (lse = -inf) and add nothing
    L, cols = T // 2, width // 2 * 64
    assert L <= cols
    tab = table[0, :2 * (width // 2)].view(2, width // 2).contiguous()
    q4, p4 = qn[:2 * L].view(2, L, H, 512), qp[:2 * L].view(2, L, H, 64)
    weights = torch.full((2, L, H), -torch.inf, device="cuda")
    weights[:, L - 2:] = 30.0
    weights[0, 5] = 20.0
    mass, mws = torch.zeros(2, cols, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens2 = torch.tensor([L, L], dtype=torch.int32, device="cuda")
    mla.mla_attn_mass(q4, p4, cache, tab, lens2, weights, 0, SCALE, 1.0, None, mass, mws)
    assert status(mws) == 0
    for b in range(2):
        rows = cache[tab[b].long()].view(-1, 576)[:L].double()
        want = torch.zeros(L, dtype=torch.float64, device="cuda")
        for i in ([5] if b == 0 else []) + [L - 2, L - 1]:
            q = torch.cat([q4[b, i], p4[b, i]], dim=-1).double()
            want[:i + 1] += torch.exp(q @ rows[:i + 1].T * SCALE - weights[b, i][:, None].double()).sum(dim=0)
        assert torch.allclose(mass[b, :L].double(), want, rtol=1e-3, atol=0)


@pytest.mark.parametrize("B", [3, 300])
@pytest.mark.parametrize("H", [16, 200])
def test_a_call_without_queries(B, H):
    import paged_mla_decode_09_gb300 as mla

    gen = generator(3)
    qn, qp = randn(gen, 5, H, 512), randn(gen, 5, H, 64)
    cache = randn(gen, 4, 64, 576)
    table = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 100, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(qn, 7.0), torch.full((5, H), 7.0, device="cuda")
    ws = torch.zeros(mla.mla_prefill_workspace_size(mla.make_prefill_dims(qn, cache, table, lens)), dtype=torch.uint8,
                     device="cuda")
    for window in (0, 30):
        mla.mla_prefill(qn, qp, cache, table, lens, cu, window, 2, SCALE, 1.0, out, lse, ws)
        assert status(ws) == 0  # no page id was looked at
        assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("Q", [1, 9])
def test_a_row_of_nan_stays_alone(Q, kv_dtype):
    import paged_mla_decode_09_gb300 as mla

    gen = generator(4)
    B, H, L = 2, 32, 500
    qn, qp = randn(gen, B, Q, H, 512), randn(gen, B, Q, H, 64)
    x = randn(gen, 16, 64, 576)
    f8 = kv_dtype != "bf16"
    cache = (x.float() * 50).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if f8 else x
    kv_scale = 0.02 if f8 else 1.0
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(B, 8)
    lens = torch.tensor([L, L - 70], dtype=torch.int32, device="cuda")
    ws = torch.zeros(mla.mla_decode_window_workspace_size(mla.make_dims(qn, cache, table)), dtype=torch.uint8,
                     device="cuda")
    outs = []
    for bad in (False, True):
        if bad:
            qn[0, 0, 5, 77] = torch.nan
            qn[1, Q - 1, 0, 3] = torch.inf
        out, lse = torch.zeros_like(qn), torch.zeros(B, Q, H, device="cuda")
        mla.mla_decode_window(qn, qp, cache, table, lens, 300, 4, SCALE, kv_scale, out, lse, ws)
        assert status(ws) == 0
        outs.append((out, lse))
    hit = torch.zeros(B, Q, H, dtype=torch.bool, device="cuda")
    hit[0, 0, 5] = hit[1, Q - 1, 0] = True
    (o0, l0), (o1, l1) = outs
    assert torch.equal(o0[~hit], o1[~hit]) and torch.equal(l0[~hit], l1[~hit])
    assert bool(o1[0, 0, 5].isnan().all()) and bool(l1[0, 0, 5].isnan())


def evict_inputs(gen, B, L, budget):
    lens = torch.randint(L // 2, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    npg = -(-L // 64)
    table = torch.randperm(B * npg, generator=gen, device="cuda").to(torch.int32).view(B, npg)
    cache = torch.randint(0, 256, (B * npg, 64, 576), generator=gen, device="cuda", dtype=torch.uint8)
    mass = torch.rand(B, npg * 64, generator=gen, device="cuda")
    return lens, table, cache, mass


def plain_evict(lens, table, cache, mass, budget, sinks, recent):
    """The rule with sorts, on the device: kept [B, budget] and the cache."""
    kept = torch.full((len(lens), budget), -1, dtype=torch.int32, device="cuda")
    out = cache.clone()
    for b, n in enumerate(lens.tolist()):
        k = min(n, budget)
        w = mass[b, :n].double()
        w[:sinks] = torch.inf
        w[max(0, n - recent):] = torch.inf
        chosen = torch.sort(torch.argsort(w, descending=True, stable=True)[:k]).values
        slots = torch.arange(k, device="cuda")
        src = slots.clone()
        hole = ~torch.isin(slots, chosen)
        src[hole] = chosen[chosen >= k]
        kept[b, :k] = src.int()
        out[table[b, slots // 64].long(), slots % 64] = cache[table[b, src // 64].long(), src % 64]
    return kept, out


def test_eviction_of_many_requests_and_a_table_slice():
    import paged_mla_decode_09_gb300 as mla

    gen = generator(5)
    B, L, budget = 3000, 180, 64
    lens, table, cache, mass = evict_inputs(gen, B, L, budget)
    want, want_cache = plain_evict(lens, table, cache, mass, budget, 3, 20)
    new_lens = [min(n, budget) for n in lens.tolist()]
    wide = torch.full((B, table.shape[1] + 3), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    table = wide[:, :table.shape[1]]
    kept = torch.zeros(B, budget, dtype=torch.int32, device="cuda")
    ws = torch.zeros(mla.mla_evict_workspace_size(B, budget), dtype=torch.uint8, device="cuda")
    mla.mla_evict(mass, None, lens, table, cache, budget, 3, 20, lens, kept, mass, None, ws)
    assert status(ws) == 0
    assert torch.equal(kept, want) and torch.equal(cache, want_cache)
    assert lens.tolist() == new_lens


def test_two_streams_of_masses_and_evictions():
    """Calls at once, each stream with its own workspace and cache."""
    import paged_mla_decode_09_gb300 as mla

    gen = generator(6)
    Q, H, B, budget = 4, 64, 3, 700
    sides = []
    for k in range(2):
        lens, table, cache, _ = evict_inputs(gen, B, 3000 + 500 * k, budget)
        cache &= 0x77  # finite codes
        qn, qp = randn(gen, B, Q, H, 512), randn(gen, B, Q, H, 64)
        lse = torch.full((B, Q, H), 12.0, device="cuda")
        mass = torch.zeros(B, table.shape[1] * 64, device="cuda")
        kept = torch.zeros(B, budget, dtype=torch.int32, device="cuda")
        mws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        ews = torch.zeros(mla.mla_evict_workspace_size(B, budget), dtype=torch.uint8, device="cuda")
        start = cache.clone()
        new = torch.zeros_like(lens)
        mo = torch.zeros_like(mass)

        def go(stream, a=(qn, qp, cache, table, lens, lse, mass, mws, kept, ews, start, new, mo)):
            qn, qp, cache, table, lens, lse, mass, mws, kept, ews, start, new, mo = a
            with torch.cuda.stream(stream):
                cache.copy_(start)
                mla.mla_attn_mass(qn, qp, cache, table, lens, lse, 0, SCALE, 0.02, None, mass, mws)
                mla.mla_evict(mass, None, lens, table, cache, budget, 4, 99, new, kept, mo, None, ews)

        go(torch.cuda.current_stream())
        assert status(mws) == 0 and status(ews) == 0
        want, want_cache = plain_evict(lens, table, start, mass, budget, 4, 99)
        assert torch.equal(kept, want) and torch.equal(cache, want_cache)
        sides.append((go, mass, kept, cache, mws, ews, [t.clone() for t in (mass, kept, cache)]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(30):
        for side, stream in zip(sides, streams):
            side[0](stream)
    for _, mass, kept, cache, mws, ews, want in sides:
        assert status(mws) == 0 and status(ews) == 0
        assert all(torch.equal(a, b) for a, b in zip((mass, kept, cache), want))


def test_graphs_that_share_a_workspace():
    """Two graphs of mass (more than 128 rows) and eviction, one behind the
    other on the same workspaces, follow their inputs."""
    import paged_mla_decode_09_gb300 as mla

    gen = generator(7)
    Q, H, B, budget = 3, 64, 4, 200
    lens, table, cache, _ = evict_inputs(gen, B, 900, budget)
    cache &= 0x77
    start, first = cache.clone(), lens.clone()
    qn, qp = randn(gen, B, Q, H, 512), randn(gen, B, Q, H, 64)
    lse = torch.full((B, Q, H), 12.0, device="cuda")
    mws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ews = torch.zeros(mla.mla_evict_workspace_size(B, budget), dtype=torch.uint8, device="cuda")
    masses = [torch.zeros(B, table.shape[1] * 64, device="cuda") for _ in range(2)]
    kepts = [torch.zeros(B, budget, dtype=torch.int32, device="cuda") for _ in range(2)]
    new, mo = torch.zeros_like(lens), torch.zeros_like(masses[0])
    graphs = []
    for mass, kept in zip(masses, kepts):
        def go():
            cache.copy_(start)
            mla.mla_attn_mass(qn, qp, cache, table, lens, lse, 0, SCALE, 0.02, None, mass, mws)
            mla.mla_evict(mass, None, lens, table, cache, budget, 4, 20, new, kept, mo, None, ews)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            go()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go()
        graphs.append(g)
    for k in range(4):
        lens.copy_(torch.where(torch.arange(B, device="cuda") % 2 == k % 2, first, first - 77))
        qn.copy_(randn(gen, *qn.shape))
        for g in graphs:
            g.replay()
        assert status(mws) == 0 and status(ews) == 0
        for b, n in enumerate(lens.tolist()):
            assert torch.equal(masses[0][b, :n], masses[1][b, :n])
        assert torch.equal(kepts[0], kepts[1])
        want, want_cache = plain_evict(lens, table, start, masses[1], budget, 4, 20)
        assert torch.equal(kepts[1], want) and torch.equal(cache, want_cache)
        q = torch.cat([qn, qp], dim=-1).double().view(B, -1, 576)
        b, n = 1, int(lens[1])
        rows = start[table[b].long()].view(-1, 576)[:n].view(torch.float8_e4m3fn).double() * 0.02
        s = q[b] @ rows.T * SCALE - 12.0
        pos = n - Q + torch.arange(Q, device="cuda").repeat_interleave(H)
        s[torch.arange(n, device="cuda")[None] > pos[:, None]] = -torch.inf
        assert torch.allclose(masses[0][b, :n].double(), torch.exp(s).sum(dim=0), rtol=1e-3, atol=1e-12)


def test_first_calls_of_a_process_are_captured():
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "first_capture_child.py")
    r = subprocess.run([sys.executable, child], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
