"""Calls given another stream than the current one: what a call makes for itself (workspace, output) belongs to
the stream that it runs on, so neither a fill that is still waiting on the current stream nor memory that the
current stream hands out again reaches it."""
import pytest

from device_logits_sampling_gb300 import kv_cache, w4

BUSY = 40_000_000  # clocks: some 20 ms


def poison(nbytes):
    """Blocks of the current stream that the next allocations of these sizes come from, full of ones."""
    import torch

    held = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in nbytes for _ in range(4)]
    torch.cuda.synchronize()
    return held


def calls():
    """Name, call (of keyword arguments) and the bytes of what it makes for itself."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(0)
    heads, q_heads, dim, page, length = 2, 8, 128, 16, 5000  # one sequence over all blocks: their joins count arrivals
    pages = -(-length // page)
    cache = kv_cache.PagedCache.empty(pages, heads, page, dim)
    for x in (cache.k, cache.v):
        x.view(torch.uint8).random_(0x20, 0x40, generator=g)
    for s in (cache.k_scale, cache.v_scale):
        s.fill_(2.0 ** -4)
    pos = torch.tensor([length - 1], dtype=torch.int32, device="cuda")
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    q = torch.randn(1, q_heads, dim, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(1, heads, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    turns = torch.from_numpy(kv_cache.rope_turns(dim)[0]).cuda()
    rope = kv_cache.Rope(turns)
    x = torch.randn(200, 1024, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(0, 256, (2000, 512), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand(2000, 8, generator=g, device="cuda").to(torch.bfloat16)
    need = cache.attend_workspace().numel()
    return [("attend", lambda **kw: kv_cache.attend(cache, q, pos, table, **kw), (need, q.numel() * 2)),
            ("append", lambda **kw: kv_cache.append(cache, k, v, pos, table, q=q, rope=rope, **kw), (q.numel() * 2,)),
            ("few", lambda **kw: w4.matvec(x[:5], w, s, **kw), (5 * 2000 * 2,)),
            ("many", lambda **kw: w4.matvec(x, w, s, **kw), (256 * 1024 * 2 + 1024, 200 * 2000 * 2))]


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(4))
def test_the_fill_of_a_workspace_comes_before_the_call(cuda_lib, which):
    """The current stream is busy: what it would fill for the call comes too late."""
    import torch

    _, call, made = calls()[which]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        del poison(made)[:]
        torch.cuda._sleep(BUSY)
        got = call(stream=side)
        side.synchronize()
        assert torch.equal(got.cpu(), want.cpu())
        torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(4))
def test_memory_is_not_handed_out_under_the_call(cuda_lib, which):
    """The call's own stream is busy: the current one allocates and fills before the call has begun."""
    import torch

    _, call, made = calls()[which]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        got = call(stream=side)
        held = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in made for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert torch.equal(got, want)
        assert all(bool((h == 0xFF).all()) for h in held)


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(4))
def test_an_output_dropped_early(cuda_lib, which):
    """The returned tensor may be read by the current stream and dropped while that has not come to it."""
    import torch

    _, call, made = calls()[which]
    want = call().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = got.clone()  # read after the sleep
    del got
    with torch.cuda.stream(side):
        held = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in made for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and len(held) > 0


@pytest.mark.gpu
def test_a_stream_that_is_current_already(cuda_lib):
    import torch

    side = torch.cuda.Stream()
    for _, call, _ in calls():
        want = call()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = call(stream=side)
        side.synchronize()
        assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(4))
def test_another_library_s_stream(cuda_lib, which):
    """A call asks no more of a stream than its handle."""
    import torch

    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    _, call, made = calls()[which]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    del poison(made)[:]
    torch.cuda._sleep(BUSY)
    got = call(stream=Handle(side))
    side.synchronize()
    assert torch.equal(got.cpu(), want.cpu())
    torch.cuda.synchronize()
