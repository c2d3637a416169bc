"""row_offsets that do not ascend from 0 to the number of rows: the sequences before the first wrong pair are stored
and attended as they would be alone; from there on nothing is stored, and every row that they do not have is NaN."""
import numpy as np
import pytest

from device_logits_sampling_gb300 import kv_cache
from oracle import kv_cache as ok
from test_kv_cache import Case, put_new

# offsets, and the sequences before the first wrong pair (six rows, three sequences)
SMALL = [([0, 4, 2, 6], 1), ([0, 2, 4, 9], 2), ([0, -2, 4, 6], 0), ([1, 2, 4, 6], 0), ([0, 2, 4, 5], 2), ([0, 6, 6, 7], 2),
         ([0, 7, 7, 6], 0), ([0, 2, 2 ** 31 - 1, 6], 1), ([0, 2, -2 ** 31, 6], 1), ([5, 3, 2, 1], 0)]


def run(c, offsets, sound, inplace=False):
    """Both calls with these offsets, against the oracle on the sound sequences alone."""
    import torch

    cache, pos, table, _ = c.device()
    T = len(c.q)
    o = torch.from_numpy(np.array(offsets, np.int32)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = c.q.cuda()
    got = kv_cache.append(cache, c.nk.cuda(), c.nv.cuda(), pos, table, q=q, q_out=q if inplace else None, rope=c.rope(),
                          row_offsets=o, err_word=err).double().cpu().numpy()
    assert int(err.item()) == kv_cache.ARC_KV_ERR_OFFSETS
    rows = int(offsets[sound]) if sound else 0
    cut = lambda x: x[:sound]  # noqa: E731
    ek, ev, eks, evs = c.k.copy(), c.v.copy(), c.ks.copy(), c.vs.copy()
    args = (cut(c.positions), cut(c.table), np.array(offsets[:sound + 1]))
    assert ok.append(ek, ev, eks, evs, c.nk.double().numpy(), c.nv.double().numpy(), *args, c.turns, 1.0, c.layout) == 0
    for g, w in ((cache.k, ek), (cache.v, ev)):
        g, zero = g.cpu().numpy(), (w & 0x7F) == 0  # the sign of a zero carries nothing
        assert np.array_equal(g & 0x7F, w & 0x7F) and np.array_equal(g[~zero], w[~zero])
    assert np.array_equal(cache.k_scale.cpu().numpy(), eks) and np.array_equal(cache.v_scale.cpu().numpy(), evs)
    eps = torch.finfo(c.dtype).eps / 2
    for b in range(sound):
        for t in range(offsets[b], offsets[b + 1]):
            x = c.q[t].double().numpy()
            want = (np.zeros_like(x) if c.positions[b] < 0 else
                    ok.rotate(x, int(c.positions[b]) + t - offsets[b], c.turns, 1.0, c.layout))
            assert (np.abs(got[t] - want) <= eps * np.abs(want) + 2.0 ** -21 * 2 * np.abs(x).max() + 2.0 ** -25).all()
    assert np.isnan(got[rows:]).all()

    err.zero_()
    out = torch.full((T, c.q_heads, c.dim), 7.0, dtype=c.dtype, device="cuda")
    kv_cache.attend(cache, c.q.cuda(), pos, table, out=out, row_offsets=o, err_word=err)
    assert int(err.item()) == kv_cache.ARC_KV_ERR_OFFSETS
    got = out.double().cpu().numpy()
    assert np.isnan(got[rows:]).all()
    if sound:
        want, spread = ok.attend(ek, ev, eks, evs, c.q.double().numpy(), *args)
        # half a step of the type, the weights' half step as fp16 and the fp32 scores
        tol = eps * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + 2.0 ** -25
        assert (np.abs(got - want)[:rows] <= tol[:rows]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("offsets,sound", SMALL)
@pytest.mark.parametrize("dim,layout,rot", [(64, "half", 64), (128, "interleaved", 64), (256, "half", 20)])
def test_three_sequences(cuda_lib, offsets, sound, dim, layout, rot):
    c = Case(61, dim, 16, 2, 6, [0, 5, 9], [2, 2, 2], "bf16", layout=layout, rot=rot, max_pages=2)
    c.table[:] = np.arange(6).reshape(3, 2)  # room for what any of the offsets may claim
    c.k, c.v = (x[:6] if len(x) >= 6 else np.concatenate([x] * 6)[:6] for x in (c.k, c.v))
    c.ks, c.vs = (x[:6] if len(x) >= 6 else np.concatenate([x] * 6)[:6] for x in (c.ks, c.vs))
    for x in (c.k, c.v):
        x[(x & 0x7F) == 0x7F] = 0x30
    for inplace in (False, True):
        run(c, offsets, sound, inplace)


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 1, 100, 255, 256, 300, 511, 512, 698, 699])
@pytest.mark.parametrize("what", ["back", "past", "garbage"])
def test_many_sequences(cuda_lib, at, what):
    """A wrong pair anywhere among more sequences than a block has threads, with anything after it."""
    rng = np.random.default_rng(at)
    n = 700
    c = Case(62, 64, 16, 1, 2, rng.integers(-1, 40, n), rng.integers(1, 4, n), "fp16", layout="interleaved")
    put_new(c)
    T = int(c.offsets[-1])
    o = c.offsets.copy()
    if what == "back":
        o[at + 1] = o[at] - 1
    elif what == "past":
        o[at + 1] = T + 1
    else:
        o[at + 1:] = rng.integers(-5, T + 5, n - at)
        o[at + 1] = o[at] - 1
    run(c, o.tolist(), at)
