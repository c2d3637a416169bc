"""attend_shared where a block of the prefix's kernel takes several chunks of a unit, and several units: references that
stay from chunk to chunk and that move between them, rings that wrap, the next unit's queries over the last one's.  More
than 152 chunks of 128 tokens (64 for heads of 256) and 256 rows (128) of a cached head.  Tolerances as in
test_attend_shared."""
import numpy as np
import pytest
from scipy.ndimage import maximum_filter1d

from oracle import kv_cache as ok
from test_attend_shared import check, run, shared_case


def settle(c, kind):
    if kind == "near":  # scores and value scales that keep their references
        c.ks[:] = 2.0 ** -9
        c.vs[:] = 2.0 ** c.rng.integers(-6, -3, c.vs.shape)
    elif kind == "apart":  # value scales that split chunks, scores that move
        c.ks[:] = 2.0 ** c.rng.integers(-9, -4, c.ks.shape)
        c.vs[:] = 2.0 ** c.rng.integers(-30, 31, c.vs.shape)
        small = c.vs[:, 0] < 1
        c.vs[:] = np.where(small, 2.0 ** c.rng.integers(-30, 0, small.shape), 2.0 ** c.rng.integers(0, 31, small.shape))[:, None]
        c.v[~small, :, :, 7] = 0
        c.v[small, :, :, 7] = 0x30
        c.v[(c.v & 0x7F) == 0x7F] = 0x30
    elif kind == "rising":  # scores that grow along the prefix, and fall again
        n = len(c.prefix)
        c.ks[:] = 2.0 ** -9
        c.ks[c.prefix] = 2.0 ** (-12 + 8 * np.sin(np.linspace(0, np.pi, n)))[:, None]
        c.vs[:] = 2.0 ** -5
    return c


def small_weights(c):
    """What weights far below those beside them may be off by, [T, q_heads, dim].  The prefix's enter as fp16, 64 tokens at
    a time: 2^-23 of the largest of the 64 at most (arc_kv.h), which lies among the 63 tokens on either side; the own
    tokens', 16 or 32 at a time, 2^-39 of the largest."""
    out = np.zeros(c.q.shape)
    for b, pos in enumerate(c.positions):
        if pos < 0:
            continue
        for h in range(c.heads):
            k, v = (ok.gather(x, s, c.table[b], pos + 1, h) for x, s in ((c.k, c.ks), (c.v, c.vs)))
            rows = slice(h * (c.q_heads // c.heads), (h + 1) * (c.q_heads // c.heads))
            s = c.q[b, rows].double().numpy() @ k.T * c.dim ** -0.5
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[b, rows] = 2.0 ** -23 * maximum_filter1d(w, 127, axis=1) @ np.abs(v)
    return out


def check_past_fp16(c):
    """Values that pass fp16's range, one token a sequence: from 65,504 + 16, half a step above its largest number, a
    rounding to nearest gives infinity."""
    got = run(c, single=True).double().cpu().numpy()
    want, spread = ok.attend(c.k, c.v, c.ks, c.vs, c.q.double().numpy(), c.positions, c.table, c.offsets)
    tol = 2.0 ** -11 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + small_weights(c) + 2.0 ** -25
    assert not np.isnan(want).any() and not np.isnan(got).any()
    past = np.isinf(got)
    assert (np.sign(got[past]) * want[past] + tol[past] >= 65520).all()
    assert (np.abs(got - want) <= tol)[~past].all(), float(np.max((np.abs(got - want) / tol)[~past]))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,heads,group,front", [(64, 16, 8, 4, 519), (128, 64, 8, 4, 130), (128, 16, 8, 2, 515),
                                                        (256, 32, 4, 3, 261), (256, 256, 4, 2, 33)])
@pytest.mark.parametrize("kind", ["near", "any", "apart", "rising"])
def test_several_chunks_a_block(cuda_lib, dim, page, heads, group, front, kind):
    c = settle(shared_case(81, dim, page, heads, group, front, [5, 200], [1, 1]), kind)
    check(c, single=True, exact_columns=kind == "apart")


@pytest.mark.gpu
@pytest.mark.parametrize("dim,heads,group,front,batch", [(64, 16, 8, 5, 500), (128, 16, 8, 9, 290), (128, 32, 5, 3, 300),
                                                         (256, 8, 8, 5, 300), (256, 16, 4, 2, 360)])
@pytest.mark.parametrize("kind", ["near", "any", "apart"])
def test_several_units_a_block(cuda_lib, dim, heads, group, front, batch, kind):
    rng = np.random.default_rng(82)
    own = [None if v < 0 else int(v) for v in rng.integers(-1, 20, batch)]
    c = settle(shared_case(82, dim, 16, heads, group, front, own, [1] * batch, "fp16"), kind)
    if kind == "apart":
        check_past_fp16(c)
    else:
        check(c, single=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,heads,group,front,batch", [(64, 8, 8, 50, 200), (128, 8, 6, 60, 170), (256, 4, 8, 40, 130)])
def test_chunks_of_several_units_and_calls_that_repeat(cuda_lib, dim, heads, group, front, batch):
    """Pieces that begin and end inside units; the same call gives the same bits."""
    import torch

    rng = np.random.default_rng(83)
    own = [int(v) for v in rng.integers(0, 60, batch)]
    c = shared_case(83, dim, 16, heads, group, front, own, [1] * batch)
    check(c, single=True)
    want = run(c, single=True)
    for _ in range(3):
        assert torch.equal(run(c, single=True), want)
