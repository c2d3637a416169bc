"""Attention within a window with first tokens that stay visible, against the fp64 oracle; tolerances as for the
attention without them (test_kv_cache)."""
import ctypes

import numpy as np
import pytest

import test_kv_cache as tk
from device_logits_sampling_gb300 import kv_cache
from oracle import kv_cache as ok
from test_kv_cache import Case, lib, put_new  # noqa: F401


def test_refusals(lib):  # noqa: F811
    def call(cache=tk.fake_cache(), step=tk.fake_step(), query=tk.fake_query(window=8), sinks=4, err=None, ws=tk.FAKE, n=1 << 30):
        at = ctypes.addressof
        return lib.arc_kv_attend_sinks(at(cache), at(step), at(query), sinks, err, ws, n, None)

    for kw, rc in tk.CACHE_REFUSALS:
        assert call(cache=tk.fake_cache(**kw)) == rc, kw
    for kw, rc in tk.STEP_REFUSALS:
        assert call(step=tk.fake_step(**kw)) == rc, kw
    assert call(query=tk.fake_query(window=-1)) == -6 and call(sinks=-1) == -6 and call(query=tk.fake_query(q_heads=6)) == -2
    for sinks, window in ((4, 8), (0, 8), (4, 0)):
        kw = dict(sinks=sinks, query=tk.fake_query(window=window))
        assert call(ws=None, **kw) == -8 and call(n=64, **kw) == -8 and call(ws=tk.FAKE + 8, **kw) == -4


def test_the_oracle_by_hand():
    """Values 1, 2, 4, 8, ... of tokens that weigh alike: 2 sinks and a window of 3."""
    k = np.zeros((2, 1, 16, 64), np.uint8)
    v = np.zeros((2, 1, 16, 64), np.uint8)
    v[:] = ok.encode(np.arange(32.0).reshape(2, 1, 16, 1))
    one = np.ones((2, 1))
    out, _ = ok.attend(k, v, one, one, np.ones((4, 1, 64)), [1, 18], np.array([[0, 1], [0, 1]]), [0, 2, 4], window=3, sinks=2)
    t = ok.TABLE[v].reshape(32, 64)[:, 0]
    want = [t[:2].mean(), t[:3].mean(), t[[0, 1, 16, 17, 18]].mean(), t[[0, 1, 17, 18, 19]].mean()]
    assert np.allclose(out[:, 0, 0], want)


def check(c, window, sinks, single=False, err_want=0, workspace=None):
    import torch

    cache, pos, table, offs = c.device()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kv_cache.attend(cache, c.q.cuda(), pos, table, row_offsets=None if single else offs, window=window, sinks=sinks,
                          err_word=err, workspace=workspace)
    torch.cuda.synchronize()
    assert int(err.item()) == err_want
    want, spread = ok.attend(c.k, c.v, c.ks, c.vs, c.q.double().numpy(), c.positions, c.table, c.offsets, None, window, sinks)
    got = got.double().cpu().numpy()
    seen = window + sinks + int(c.news.max())
    vmax = float(448.0 * c.vs.max())
    eps = torch.finfo(c.dtype).eps / 2
    tol = eps * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + 2.0 ** -25 * seen * vmax + 2.0 ** -25
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bad = ~(np.abs(got - want) <= tol) & ~np.isnan(want)
    assert not bad.any(), (np.argwhere(bad)[:5], float(np.nanmax(np.abs(got - want) / tol)))


def forget(c, window, sinks):
    """Takes the pages that no new token sees out of the table, and fills them with NaN."""
    for b in range(len(c.positions)):
        p = int(c.positions[b])
        if p < 0:
            continue
        lo, hi = -(-sinks // c.page), max(0, p + 1 - window) // c.page
        for j in range(lo, hi):
            if c.table[b, j] >= 0:
                c.k[c.table[b, j]] = c.v[c.table[b, j]] = 0x7F
            c.table[b, j] = -1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,page,heads,group,window,sinks", [
    (64, 16, 2, 1, 20, 1), (64, 64, 1, 4, 100, 33), (128, 16, 2, 8, 1, 4), (128, 64, 3, 5, 65, 64), (128, 256, 1, 16, 300, 17),
    (256, 32, 2, 2, 40, 50), (256, 16, 1, 9, 16, 16), (64, 32, 1, 17, 31, 31), (64, 16, 1, 8, 33, 16), (64, 16, 1, 2, 50, 48),
    (128, 32, 1, 3, 2000, 3), (128, 32, 1, 3, 4, 5000)])
def test_one_token_each(cuda_lib, dtype, dim, page, heads, group, window, sinks):
    """Positions on every side of the sinks, the window's start and the pages' ends; pages that nobody sees are gone."""
    pos = [0, 1, 14, 15, 16, 17, 31, 32, 63, 64, 127, 130, 255, -1, 300, 511, 777]
    c = Case(41, dim, page, heads, heads * group, pos, [1] * len(pos), dtype)
    put_new(c)
    forget(c, window, sinks)
    check(c, window, sinks, single=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,heads,group,window,sinks", [
    (64, 16, 2, 4, 7, 1), (128, 64, 1, 1, 64, 10), (128, 32, 2, 5, 33, 70), (256, 16, 1, 3, 1, 16), (64, 32, 1, 8, 16, 30),
    (128, 16, 1, 16, 100, 4)])
def test_several_tokens(cuda_lib, dim, page, heads, group, window, sinks):
    pos, news = [0, 3, 15, 100, 0, 250, -1, 60, 400], [1, 5, 17, 8, 33, 2, 3, 0, 90]
    c = Case(42, dim, page, heads, heads * group, pos, news, "bf16")
    put_new(c)
    forget(c, window, sinks)
    check(c, window, sinks)


@pytest.mark.gpu
def test_long_and_many(cuda_lib):
    c = Case(43, 128, 64, 2, 8, [20000], [1], "bf16", fill=False)
    for x in (c.k, c.v):
        x[(x & 0x7F) == 0x7F] = 0x30
    forget(c, 5000, 100)
    check(c, 5000, 100, single=True)
    check(c, 20, 4, single=True)
    rng = np.random.default_rng(44)
    n = 1500
    c = Case(44, 64, 16, 1, 4, rng.integers(-1, 90, n), np.ones(n, int), "fp16")
    put_new(c)
    forget(c, 17, 5)
    check(c, 17, 5, single=True)


@pytest.mark.gpu
def test_without_a_window_or_sinks_it_is_the_plain_call(cuda_lib):
    import torch

    c = Case(45, 128, 16, 2, 6, [30, 50, 200, 16], [1] * 4, "bf16")
    put_new(c)
    cache, pos, table, _ = c.device()
    q = c.q.cuda()
    call = lambda **kw: kv_cache.attend(cache, q, pos, table, **kw)  # noqa: E731
    assert torch.equal(call(sinks=7), call()) and torch.equal(call(sinks=0, window=9), call(window=9))
    assert torch.equal(call(sinks=1000, window=9), call())  # everything is a first token
    assert torch.equal(call(sinks=2 ** 31 - 1, window=2 ** 31 - 1), call())


@pytest.mark.gpu
def test_nan_reaches_those_that_see_it(cuda_lib):
    """A NaN value under the sinks reaches every row; one that the window has left, only the rows before."""
    c = Case(46, 64, 16, 1, 2, [60], [4], "bf16")
    put_new(c)
    page = lambda t: (c.table[0, t // 16], 0, t % 16)  # noqa: E731
    c.v[page(2)][5] = 0x7F  # a sink
    c.v[page(42)][9] = 0x7F  # seen by positions up to 61 through a window of 20
    c.v[page(3)][11] = 0x7F  # just past the sinks
    cache, pos, table, offs = c.device()
    got = kv_cache.attend(cache, c.q.cuda(), pos, table, row_offsets=offs, window=20, sinks=3).float().cpu().numpy()
    nan = np.zeros_like(got, dtype=bool)
    nan[:, :, 5] = True
    nan[:2, :, 9] = True
    assert np.array_equal(np.isnan(got), nan)


@pytest.mark.gpu
def test_bad_pages(cuda_lib):
    """A bad page under the sinks spoils its sequence; one between sinks and window is not looked at."""
    c = Case(47, 64, 16, 2, 4, [30, 90, 90], [1] * 3, "bf16")
    put_new(c)
    c.table[1, 0] = len(c.k)
    c.table[2, 2] = -7
    check(c, 20, 4, single=True, err_want=1)


@pytest.mark.gpu
def test_a_stream_of_steps_replayed(cuda_lib):
    """Tokens appended and attended to step by step, pages between sinks and window given back on the way: each
    replayed step is the oracle's attention over what is visible."""
    import torch

    window, sinks, page, steps = 24, 5, 16, 90
    pages = -(-steps // page)
    c = Case(48, 64, page, 2, 4, [0, 0], [1, 1], "bf16", max_pages=pages)
    c.k, c.v = (np.zeros((2 * pages, 2, page, 64), np.uint8) for _ in range(2))
    c.ks, c.vs = np.ones((2 * pages, 2)), np.ones((2 * pages, 2))
    c.table = np.arange(2 * pages, dtype=np.int32).reshape(2, pages)
    cache, pos, table, _ = c.device()
    ws, rope, x = cache.attend_workspace(), c.rope(), torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        q = kv_cache.append(cache, x[:, 4:6], x[:, 6:8], pos, table, q=x[:, :4], rope=rope, err_word=err)
        o = kv_cache.attend(cache, q, pos, table, workspace=ws, window=window, sinks=sinks, err_word=err)
        pos.add_(1)
        return q, o

    step()
    pos.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o = step()
    pos.zero_()
    for i in range(steps):
        x.copy_(torch.randn(x.shape, device="cuda"))
        gone = max(0, i + 1 - window) // page
        if gone > 1:  # page 0 has the sinks
            table[:, 1:gone] = -1
        graph.replay()
        host = [t.cpu().numpy() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)]
        want, spread = ok.attend(*host, q.double().cpu().numpy(), [i, i], table.cpu().numpy(), [0, 1, 2], None, window, sinks)
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + 2.0 ** -18
        assert (np.abs(o.double().cpu().numpy() - want) <= tol).all()
    assert int(err) == 0
