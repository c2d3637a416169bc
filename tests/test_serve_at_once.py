"""Calls of several streams at once, each with a workspace of its own, eager and replayed: the same bits as one after another.
And prefixes that name a page more than once, or one that a sequence also has behind the prefix."""
import numpy as np
import pytest

from device_logits_sampling_gb300 import edit, kv_cache, norm
from test_attend_shared import check, shared_case


@pytest.mark.gpu
def test_streams_at_once(cuda_lib):
    import torch

    calls = []
    for seed, dim, heads, group, front, batch in ((111, 128, 8, 4, 70, 40), (112, 64, 4, 8, 90, 70), (113, 256, 4, 2, 40, 30)):
        c = shared_case(seed, dim, 16, heads, group, front, [i * 7 % 90 for i in range(batch)], [1] * batch)
        cache, pos, table, _ = c.device()
        prefix, q = torch.from_numpy(c.prefix.astype(np.int32)).cuda(), c.q.cuda()
        ws, plain = cache.shared_workspace(batch, heads * group), cache.attend_workspace()
        out, near = torch.empty_like(q), torch.empty_like(q)

        def call(cache=cache, q=q, pos=pos, table=table, prefix=prefix, ws=ws, plain=plain, out=out, near=near):
            kv_cache.attend_shared(cache, q, pos, table, prefix, out=out, workspace=ws)
            kv_cache.attend(cache, q, pos, table, out=near, workspace=plain, window=200, sinks=20)

        calls.append((call, (out, near)))
    x, y = (torch.randn(1300, 5120, device="cuda").to(torch.bfloat16) for _ in range(2))
    h, n = torch.empty_like(x), torch.empty_like(x)
    calls.append((lambda: norm.join(x, y, h=h, n=n), (h, n)))
    z, mask = torch.randn(64, 50003, device="cuda"), torch.randint(-(1 << 31), (1 << 31) - 1, (64, 1563), device="cuda").to(torch.int32)
    e = torch.empty_like(z)
    calls.append((lambda: edit.edit_logits(z, out=e, allowed=mask), (e,)))
    want = []
    for call, outs in calls:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in calls]
    graphs = []
    for call, _ in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for run in ([c for c, _ in calls], [g.replay for g in graphs]):
        for _, outs in calls:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for f, s in zip(run, streams):
                with torch.cuda.stream(s):
                    f()
        torch.cuda.synchronize()
        for (_, outs), w in zip(calls, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, w))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,front", [(64, 16, 30), (128, 64, 9), (256, 32, 11)])
def test_a_page_named_twice(cuda_lib, dim, page, front):
    c = shared_case(114, dim, page, 2, 3, front, [40, 100, 7], [1] * 3)
    c.prefix[1::3] = c.prefix[0]
    c.table[:, :front] = c.prefix
    c.table[1, front] = c.prefix[2]  # a whole page behind the prefix
    check(c, single=True)
