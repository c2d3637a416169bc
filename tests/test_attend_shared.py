"""Attention of sequences that share a prefix against the fp64 oracle over their whole tables; tolerances as for the
attention of each by itself (test_kv_cache): the weights' half step of fp16 and the fp32 scores."""
import ctypes

import numpy as np
import pytest

import test_kv_cache as tk
from device_logits_sampling_gb300 import kv_cache
from oracle import kv_cache as ok
from test_kv_cache import Case, lib, put_new  # noqa: F401


def test_refusals(lib):  # noqa: F811
    at = ctypes.addressof

    def call(cache=tk.fake_cache(), step=tk.fake_step(), query=tk.fake_query(), prefix=tk.FAKE, pages=2, err=None, ws=tk.FAKE,
             n=1 << 40):
        return lib.arc_kv_attend_shared(at(cache), at(step), at(query), prefix, pages, err, ws, n, None)

    for kw, rc in tk.CACHE_REFUSALS:
        assert call(cache=tk.fake_cache(**kw)) == rc, kw
    for kw, rc in tk.STEP_REFUSALS:
        assert call(step=tk.fake_step(**kw)) == rc, kw
    for kw, rc in [(dict(prefix=None), -1), (dict(pages=0), -2), (dict(pages=-1), -2), (dict(pages=6), -2), (dict(prefix=tk.FAKE + 2), -4),
                   (dict(query=tk.fake_query(window=8)), -6), (dict(query=tk.fake_query(q_heads=6)), -2),
                   (dict(ws=None), -8), (dict(n=0), -8), (dict(ws=tk.FAKE + 8), -4), (dict(err=tk.FAKE + 1), -4),
                   (dict(step=tk.fake_step(T=1 << 20, row_offsets=tk.FAKE)), -2)]:
        assert call(**kw) == rc, kw
    size = lib.arc_kv_attend_shared_workspace_bytes
    cache = tk.fake_cache()
    need = size(at(cache), 3, 8)
    assert need > 0 and call(n=need - 1) == -8
    assert size(at(cache), 0, 8) == 0 and size(at(cache), 3, 6) == 0 and size(at(cache), 1 << 20, 8) == 0
    assert size(at(tk.fake_cache(head_dim=96)), 3, 8) == 0 and size(None, 3, 8) == 0


def test_python_refusals():
    import torch

    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    s = torch.ones(4, 2)
    cache = kv_cache.PagedCache(k, k.clone(), s, s.clone())
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pos, table, pre = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for kw in (dict(q=x[:2]), dict(q=x[..., :32]), dict(prefix=table), dict(prefix=torch.zeros(4, dtype=torch.int32)[::2]), dict()):
        with pytest.raises(ValueError):  # the last: host tensors
            kv_cache.attend_shared(cache, **{**dict(q=x, positions=pos, page_table=table, prefix=pre), **kw})
    for kw in (dict(prefix=pre.long()), dict(q=x.float())):
        with pytest.raises(TypeError):
            kv_cache.attend_shared(cache, **{**dict(q=x, positions=pos, page_table=table, prefix=pre), **kw})


def shared_case(seed, dim, page, heads, group, front, own, news, dtype="bf16", **kw):
    """Sequences that hold `own` tokens before the new ones behind a prefix of `front` pages (None: parked)."""
    pos = [-1 if o is None else front * page + o for o in own]
    c = Case(seed, dim, page, heads, heads * group, pos, news, dtype, **kw)
    first = next(b for b, p in enumerate(pos) if p >= 0)
    c.prefix = c.table[first, :front].copy()
    c.table[:, :front] = c.prefix
    put_new(c)
    return c


def run(c, single=False, hide=True, **kw):
    import torch

    cache, pos, table, offs = c.device()
    if hide:
        table[:, : len(c.prefix)] = -1  # not read
    prefix = torch.from_numpy(c.prefix.astype(np.int32)).cuda()
    return kv_cache.attend_shared(cache, kw.pop("q", c.q.cuda()), pos, table, prefix, row_offsets=None if single else offs, **kw)


def check(c, single=False, err_want=0, exact_columns=False, **kw):
    import torch

    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(c, single, err_word=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == err_want
    want, spread = ok.attend(c.k, c.v, c.ks, c.vs, c.q.double().numpy(), c.positions, c.table, c.offsets, kw.get("scale"))
    got = got.double().cpu().numpy()
    n = max(1, int((c.positions + c.news).max()))
    eps = torch.finfo(c.dtype).eps / 2
    lost = 0.0 if exact_columns else 2.0 ** -25 * n * 448.0 * float(c.vs.max())
    tol = eps * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + lost + 2.0 ** -25
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bad = ~(np.abs(got - want) <= tol) & ~np.isnan(want)
    assert not bad.any(), (np.argwhere(bad)[:5], float(np.nanmax(np.abs(got - want) / tol)))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,heads,group,front", [
    (64, 16, 2, 1, 1), (64, 64, 1, 4, 3), (64, 16, 2, 8, 40), (128, 16, 1, 4, 9), (128, 64, 3, 5, 2), (128, 256, 1, 16, 3),
    (128, 128, 2, 8, 5), (128, 32, 2, 40, 13), (256, 16, 1, 2, 5), (256, 32, 2, 3, 9), (256, 256, 1, 9, 2), (64, 128, 1, 17, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_token_each(cuda_lib, dtype, dim, page, heads, group, front):
    """Own parts of every length around steps and pages; prefixes that end inside a tile."""
    own = [0, 1, 14, 15, 16, 17, 31, 63, 64, 130, None, 255, 300]
    check(shared_case(61, dim, page, heads, group, front, own, [1] * len(own), dtype), single=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,heads,group,front", [(64, 16, 2, 4, 9), (128, 64, 1, 1, 2), (128, 32, 2, 5, 11), (256, 16, 1, 3, 17)])
def test_several_tokens(cuda_lib, dim, page, heads, group, front):
    own, news = [0, 3, 15, 100, 0, 250, None, 60], [1, 5, 17, 8, 33, 2, 3, 0]
    check(shared_case(62, dim, page, heads, group, front, own, news))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,batch,group,front", [(64, 300, 4, 33), (128, 129, 2, 20), (128, 700, 1, 4), (256, 150, 2, 10)])
def test_many_rows(cuda_lib, dim, batch, group, front):
    """More rows than a unit has; units that begin inside a block's piece."""
    rng = np.random.default_rng(63)
    own = [None if v < 0 else int(v) for v in rng.integers(-1, 30, batch)]
    check(shared_case(63, dim, 16, 2, group, front, own, [1] * batch, "fp16"), single=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,front", [(128, 64, 300), (64, 16, 700), (256, 32, 301)])
def test_long_prefix(cuda_lib, dim, page, front):
    c = shared_case(64, dim, page, 1, 4, front, [5, 200], [1, 1])
    check(c, single=True)
    check(c, single=True, scale=-0.02)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_value_scales_far_apart(cuda_lib, dim):
    """Pages of 16 tokens whose value scales differ by up to 2^60, in and behind the prefix: columns that only the
    small pages fill keep their values."""
    c = shared_case(65, dim, 16, 1, 3, 37, [40, 3, 90], [1] * 3)
    c.vs[:] = 2.0 ** c.rng.integers(-30, 31, c.vs.shape)
    c.ks[:] = 2.0 ** -8
    small = c.vs[:, 0] < 1
    c.v[~small, :, :, 7] = 0
    c.v[small, :, :, 7] = 0x30
    for x in (c.v,):
        x[(x & 0x7F) == 0x7F] = 0x30
    check(c, single=True, exact_columns=True)
    c.vs[:] = (c.vs * 1.37).astype(np.float32)
    check(c, single=True, exact_columns=True)


@pytest.mark.gpu
def test_extreme_scores(cuda_lib):
    """One token takes all the weight, in the prefix or behind it; all weigh alike."""
    import torch

    for factor in (200.0, 0.0, 1e-30):
        c = shared_case(66, 128, 16, 1, 3, 20, [0, 40, 77], [1] * 3)
        c.ks[:] = 2.0 ** -6
        c.q = (c.q.float() * factor).to(torch.bfloat16)
        if factor > 1:
            c.q = torch.round(c.q.float() / 64).mul(64).to(torch.bfloat16)  # few bits: exact products
        check(c, single=True)


@pytest.mark.gpu
def test_nan_values_and_queries(cuda_lib):
    import torch

    c = shared_case(67, 64, 16, 1, 2, 10, [3, 20, None], [2, 1, 1])
    c.v[c.prefix[4], 0, 3, 5] = 0xFF  # a NaN in the prefix: everyone's
    p = c.table[0, 10]
    c.v[p, 0, 4, 9] = 0x7F  # sequence 0's last token
    c.v[p, 0, 5:] = c.k[p, 0, 5:] = 0x7F  # behind it
    c.q[2, 1, 3] = float("nan")
    got = run(c).float().cpu().numpy()
    nan = np.zeros_like(got, dtype=bool)
    nan[:3, :, 5] = True
    nan[1, :, 9] = True
    nan[2, 1] = True
    assert np.array_equal(np.isnan(got), nan) and not got[3].any() and torch.isfinite(torch.from_numpy(got[3])).all()


@pytest.mark.gpu
def test_wrong_pages_positions_and_offsets(cuda_lib):
    import torch

    c = shared_case(68, 64, 16, 2, 4, 3, [30, 50, 16], [1] * 3)
    c.table[1, 3] = len(c.k)
    check(c, single=True, err_want=1)
    c = shared_case(68, 64, 16, 2, 4, 3, [30, 50, 16], [1] * 3)
    c.prefix[1] = -1
    c.table[:, 1] = -1
    check(c, single=True, err_want=1)
    c = shared_case(69, 128, 16, 2, 4, 3, [30, 50, 16], [1, 2, 1])
    c.positions[1] = 3 * 16 - 1  # inside the prefix
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(c, err_word=err).float().cpu()
    assert int(err) == 2 and torch.isnan(got[1:3]).all() and torch.isfinite(got[[0, 3]]).all()
    c = shared_case(69, 128, 16, 2, 4, 3, [30, 50, 16], [1, 2, 1])
    c.max_pages -= 1
    c.table = np.ascontiguousarray(c.table[:, :-1])
    err.zero_()
    got = run(c, err_word=err).float().cpu()
    assert int(err) == 2 and torch.isnan(got[1:3]).all() and torch.isfinite(got[[0, 3]]).all()
    c = shared_case(70, 64, 16, 1, 2, 3, [3, 5, 9], [2, 2, 2])
    want = run(c)
    c.offsets = np.array([0, 2, 1, 6], np.int32)
    err.zero_()
    got = run(c, err_word=err)
    assert int(err) == 8 and torch.isnan(got[2:]).all() and torch.equal(got[:2], want[:2])


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_memory_workspace_streams_and_graphs(cuda_lib, dim):
    """Strided queries and outputs, head-major caches; a workspace that serves call after call, also one made for more
    tokens; another stream; a captured call."""
    import torch

    c = shared_case(71, dim, 16, 2, 3, 21, [30, 50, 400, 16], [1] * 4, head_major=True)
    check(c, single=True)
    c.head_major = False
    want = run(c, single=True)
    for strided in (1, 8):
        wide = torch.full((4, 7, dim + strided), 7.0, dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(wide, 7.0)
        wide[:, 1:, strided:] = c.q.cuda()
        run(c, single=True, q=wide[:, 1:, strided:], out=out[:, 1:, strided:])
        assert torch.equal(out[:, 1:, strided:], want)
        assert (out[:, 0] == 7).all() and (out[:, :, :strided] == 7).all()
    cache, pos, table, _ = c.device()
    prefix, q = torch.from_numpy(c.prefix.astype(np.int32)).cuda(), c.q.cuda()
    ws = cache.shared_workspace(9, 6)
    call = lambda **kw: kv_cache.attend_shared(cache, q, pos, table, prefix, **kw)  # noqa: E731
    for _ in range(3):
        assert torch.equal(call(workspace=ws), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got.cpu(), want.cpu())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(workspace=ws)
    for step in range(3):
        pos.add_(-1)
        if step:  # (one token less may weigh nothing: other queries, too)
            q.copy_(torch.randn(q.shape, device="cuda"))
        graph.replay()
        assert torch.equal(out, call())
    assert not torch.equal(out, want)


@pytest.mark.gpu
def test_one_query_of_each_row_alone(cuda_lib):
    """Rows do not depend on what else is in the batch: each sequence alone gives what it gives among the others,
    to the roundings of parts cut elsewhere."""
    import torch

    c = shared_case(72, 128, 32, 2, 4, 30, [0, 33, 64, 100], [1] * 4)
    cache, pos, table, _ = c.device()
    prefix, q = torch.from_numpy(c.prefix.astype(np.int32)).cuda(), c.q.cuda()
    full = kv_cache.attend_shared(cache, q, pos, table, prefix).float()
    for b in range(4):
        one = kv_cache.attend_shared(cache, q[b:b + 1], pos[b:b + 1], table[b:b + 1], prefix).float()
        plain = kv_cache.attend(cache, q[b:b + 1], pos[b:b + 1], table[b:b + 1]).float()
        scale = full[b].abs().max()
        assert (one[0] - full[b]).abs().max() <= 2.0 ** -7 * scale and (plain[0] - full[b]).abs().max() <= 2.0 ** -7 * scale
