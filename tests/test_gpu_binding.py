"""The binding's calls of a speculative step take exactly the tensors that the
library expects: every argument in turn is replaced by one of another type,
shape, layout or device, and the call raises before anything is enqueued."""
import pytest

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


def z(*shape, t=torch.int32):
    return torch.zeros(shape, dtype=t, device="cuda")


def calls():
    """name -> (function, arguments, places of the tensors, places that may be None)."""
    import paged_mla_decode_09_gb300 as mla

    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    B, T, H, V, cols = 2, 5, 3, 40, 4
    cu = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 70, dtype=torch.int32, device="cuda")
    table = torch.arange(B * cols, dtype=torch.int32, device="cuda").view(B, cols)
    cache = z(10, 64, 576, t=bf)
    parents = torch.tensor([-1, 0, -1, 0, 1], dtype=torch.int32, device="cuda")
    ws = z(64 << 20, t=u8)
    refs = torch.ones(10, dtype=torch.int32, device="cuda")
    return {
        "tree": (mla.mla_decode_tree, [z(T, H, 512, t=bf), z(T, H, 64, t=bf), cache, table, lens, cu, parents, 0.1, 1.0,
                                       z(T, H, 512, t=bf), z(T, H, t=f32), ws], (0, 1, 2, 3, 4, 5, 6, 9, 10, 11), ()),
        "commit": (mla.mla_tree_commit, [z(2, 10, 64, 576, t=u8), table, lens, cu, z(B, 3), z(B), z(B), z(1)],
                   (0, 1, 2, 3, 4, 5, 6, 7), ()),
        "verify": (mla.mla_verify, [torch.full((T, V), 1 / V, device="cuda"), torch.full((T, V), 1 / V, device="cuda"), z(T),
                                    parents, cu, z(T, t=f32), z(B, t=f32), z(B, 3), z(B, 3), z(B), z(1)],
                   tuple(range(11)), (1,)),
        "resize": (mla.mla_page_resize, [lens, table, refs, table.clone(), refs.clone(), ws], (0, 1, 2, 3, 4, 5), ()),
        "fork": (mla.mla_page_fork, [z(3), lens, table, refs, cache, z(3, cols), refs.clone(), ws], tuple(range(8)), ()),
        "rope": (mla.mla_rope_pack, [mla.mla_rope_plan(64), z(T, H, 64, t=bf), z(T, 576, t=bf), z(T), table, lens, cu, 1.0,
                                     z(T, H, 64, t=bf), cache, z(1)], (1, 2, 3, 4, 5, 6, 8, 9, 10), (3,)),
    }


LOOSE = {"tree": {11}, "commit": {7}, "verify": {10}, "resize": {5}, "fork": {7}, "rope": {10}}  # any shape will do


def others(t, loose):
    """Tensors that are not like t."""
    yield t.cpu()
    other = {torch.bfloat16: torch.float16, torch.float32: torch.float64, torch.int32: torch.int64, torch.uint8: torch.int8}
    if not (loose and t.dtype == torch.uint8):  # (a workspace is bytes of any type)
        yield t.to(other[t.dtype])
    if loose:
        if t.dim() == 1 and t.numel() > 2 and t.dtype == torch.uint8:
            yield t[::2]
        else:
            yield t[:0]
        return
    yield t[None]
    yield t[:-1]
    yield torch.cat([t, t[:1]])
    if t.shape[-1] > 1 and t.dim() > 1:
        yield t.transpose(-1, -2).contiguous().transpose(-1, -2)
        yield t[..., :-1].contiguous()


def fits(name, k, bad, good):
    if not torch.is_tensor(bad) or not bad.is_cuda or bad.dtype != good.dtype or not bad.is_contiguous():
        return False
    if (name, k) in (("commit", 0), ("fork", 4)):
        return bad.dim() in (3, 4) and bad.shape[-2:] == (64, 576) and (name == "commit" or bad.shape[-3] == 10)
    if (name, k) in (("tree", 2), ("rope", 9)):
        return bad.dim() == 3 and bad.shape[1:] == (64, 576)
    if (name, k) in (("tree", 3), ("commit", 1), ("commit", 4), ("rope", 4)):
        return bad.dim() == 2 and bad.shape[0] == 2
    return False


@pytest.mark.parametrize("name", ["tree", "commit", "verify", "resize", "fork", "rope"])
def test_every_argument_is_looked_at(name):
    import paged_mla_decode_09_gb300 as mla

    call, args, places, optional = calls()[name]
    call(*args)  # as it should be
    torch.cuda.synchronize()
    for k in places:
        for bad in [None, 3, *others(args[k], k in LOOSE[name])]:
            if bad is None and k in optional:
                continue
            if fits(name, k, bad, args[k]):
                continue  # another number of pages, layers or columns is another call
            try:
                call(*args[:k], bad, *args[k + 1:])
            except (ValueError, TypeError, AttributeError, mla.MlaError):
                continue
            raise AssertionError((name, k, bad if not torch.is_tensor(bad) else (bad.shape, bad.stride(), bad.dtype, bad.device)))
    with pytest.raises((ValueError, TypeError, AttributeError)):
        call(*args, stream=3)
    call(*args, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    call(*args)
    torch.cuda.synchronize()


def test_rope_takes_a_plan_only():
    call, args, _, _ = calls()["rope"]
    for plan in (None, 3, b"x" * 271, b"x" * 16, object()):
        with pytest.raises(TypeError):
            call(plan, *args[1:])


@pytest.mark.parametrize("name", ["tree", "commit", "verify", "resize", "fork", "rope"])
def test_other_threads_run_while_a_launch_waits(name):
    """Calls behind a kernel of a good half second: the stream's queue fills up
    and launches wait for it, and meanwhile this thread has to get on."""
    import threading
    import time

    call, args, _, _ = calls()[name]
    call(*args)
    torch.cuda.synchronize()
    took = []

    def enqueue():
        begin = time.perf_counter()
        for _ in range(4000):
            call(*args)
        took.append(time.perf_counter() - begin)

    torch.cuda._sleep(1_500_000_000)  # cycles, at 2 GHz or less
    other = threading.Thread(target=enqueue)
    longest, last = 0.0, time.perf_counter()
    other.start()
    while other.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        longest, last = max(longest, now - last), now
    other.join()
    torch.cuda.synchronize()
    assert took[0] > 0.5  # the queue was full
    assert longest < 0.2
